// Host side of the Newton-Schulz group: layout, tile lists, and the launches of one call.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <functional>
#include <queue>

#include "ns.h"

namespace psgd {
int ns_x0_tile();

namespace {

inline int64_t rup(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

constexpr int kCus = 256;

// One candidate item of a tile list.
struct Item {
  Work w;
  double cost;                           // microseconds on a CU of its own
};

// Cost model of a product list, in microseconds, fitted to runs of 13 groups in each tile width.
//   stage   one stage of 32 k of a tile, on a chip that is idle but for it
//   full    the same on a full chip, which runs at its power limit; in between by the share of CUs
//           that have an item
//   fixed, fixed_update  what a tile costs beside its stages (the update reads and writes X)
// On a full chip 256-wide tiles do 1.6 times the work per microsecond of 128-wide ones and 2.4 times
// that of 64-wide ones (A of four 2480 x 2480 in 61, 72 and 100 us); where there are few tiles the
// narrow ones finish first (A of 496 x 3968, unsplit: 62, 27 and 18 us; its update 16, 9.1 and 8.7).
// Accurate products (two stages per 32 k, three products for two stages' loads) run at the MFMA's
// pace from 128-wide tiles on (the same A: 221 and 252 us); 256-wide ones would not hold both halves
// in registers.
struct TileCost { int tile; double stage, full, fixed, fixed_update; };
constexpr TileCost kFast[] = {{64, 0.12, 0.11, 0.7, 0.8}, {128, 0.18, 0.29, 1.5, 2.5}, {256, 0.43, 0.75, 6.0, 7.0}};
constexpr TileCost kAccurate[] = {{64, 0.145, 0.14, 0.7, 1.0}, {128, 0.29, 0.37, 3.0, 4.0}};
constexpr double kLaunch = 4.0;              // a second, dependent launch
constexpr double kMemory = 4.0e6;            // bytes per microsecond of partial sums

// Time of a list whose items go, longest first, to the CU with the least work.
double makespan(std::vector<double> cost) {
  std::sort(cost.begin(), cost.end(), std::greater<double>());
  std::vector<double> start(kCus, 0.0);
  std::priority_queue<double, std::vector<double>, std::greater<double>> cus(std::greater<double>(), std::move(start));
  double last = 0.0;
  for (double c : cost) {
    const double t = cus.top() + c;
    cus.pop();
    cus.push(t);
    last = std::max(last, t);
  }
  return last;
}

// The list in the order xcd_remap deals it out: XCD x walks the x-th eighth, padded to the longest.
// Items of one cost are dealt to the XCDs in contiguous runs, since neighbours share operand rows in
// an XCD's L2, as many to each as evens out the XCDs' work; longer items come first. (Four
// resblocks' A, row-major: runs 192 us, item by item to the first free CU 222 us, where half of the XCDs had
// all of the second round.)
std::vector<Work> spread(const std::vector<Item>& items) {
  std::vector<int> idx(items.size());
  for (size_t i = 0; i < idx.size(); ++i) idx[i] = (int)i;
  std::stable_sort(idx.begin(), idx.end(), [&](int a, int b) { return items[a].cost > items[b].cost; });
  std::vector<std::vector<Work>> seg(kXcds);
  double load[kXcds] = {};
  for (size_t beg = 0; beg < idx.size();) {
    size_t end = beg;
    while (end < idx.size() && items[idx[end]].cost == items[idx[beg]].cost) ++end;
    int quota[kXcds] = {};
    for (size_t i = beg; i < end; ++i) {
      int x = 0;
      for (int y = 1; y < kXcds; ++y) if (load[y] < load[x]) x = y;
      load[x] += items[idx[i]].cost;
      ++quota[x];
    }
    for (int x = 0; x < kXcds; ++x)
      for (int k = 0; k < quota[x]; ++k) seg[x].push_back(items[idx[beg++]].w);
  }
  size_t per = 0;
  for (const auto& s : seg) per = std::max(per, s.size());
  std::vector<Work> out;
  for (auto& s : seg) {
    s.resize(per, Work{-1, 0, 0, 0});
    out.insert(out.end(), s.begin(), s.end());
  }
  return out;
}

struct Planned {
  int tile = 0;
  std::vector<Work> work, reduce;
  int64_t slots = 0;
  double time = 0.0;
};

// Tiles of one product stage.
int64_t tile_count(const std::vector<NsMat>& mats, NsStage st, int tile) {
  int64_t n = 0;
  for (const NsMat& d : mats) {
    const int64_t ns = (d.s + tile - 1) / tile, nl = (d.l + tile - 1) / tile;
    n += st == NS_UPDATE ? ns * nl : ns * (ns + 1) / 2;
  }
  return n;
}

// The tiles of one product stage, `tile` wide, in an order in which neighbours share operands:
// blocks of up to 8 x 8 tiles of the lower triangle (A and B), or the row tiles over one column panel
// of X (the update).
std::vector<Work> tiles_of(const std::vector<NsMat>& mats, NsStage st, int tile) {
  std::vector<Work> w;
  for (int i = 0; i < (int)mats.size(); ++i) {
    const int ns = (mats[i].s + tile - 1) / tile, nl = (mats[i].l + tile - 1) / tile;
    if (st == NS_UPDATE) {
      for (int a = 0; a < nl; ++a)
        for (int b = 0; b < ns; ++b) w.push_back(Work{i, a * tile, b * tile, -1});
      continue;
    }
    const int side = ns <= 8 ? ns : 4;
    for (int a0 = 0; a0 < ns; a0 += side)
      for (int b0 = 0; b0 <= a0; b0 += side)
        for (int a = a0; a < std::min(ns, a0 + side); ++a)
          for (int b = b0; b < std::min(a + 1, b0 + side); ++b) w.push_back(Work{i, a * tile, b * tile, -1});
  }
  return w;
}

// Choose the tile width and the split of K that the cost model expects to finish first. Splitting
// gives a list of few long tiles (A is s x s over K = l) enough items to fill the CUs, or evens out
// a last round that would fill part of them; it costs the partial sums' way through memory and a
// second launch.
Planned plan_list(const std::vector<NsMat>& mats, NsStage st, bool accurate) {
  Planned best;
  const int kinds = accurate ? 2 : 3;
  for (int kind = 0; kind < kinds; ++kind) {
    const TileCost& tc = accurate ? kAccurate[kind] : kFast[kind];
    if (kind + 1 < kinds && tile_count(mats, st, tc.tile) > 64 * kCus) continue;   // far past what narrow tiles are for
    const std::vector<Work> w = tiles_of(mats, st, tc.tile);
    const int n = (int)w.size();
    const double fixed = st == NS_UPDATE ? tc.fixed_update : tc.fixed;
    const double tile_bytes = 4.0 * tc.tile * tc.tile;
    auto stages = [&](const Work& x) { return ns_stages(st == NS_GRAM ? mats[x.mat].l : mats[x.mat].s, accurate); };
    double total = 0.0;
    for (const Work& x : w) total += stages(x);
    // tiles of more than `limit` stages are split, but for the first `whole` of the list
    auto consider = [&](double limit, int whole) {
      std::vector<Item> items;
      std::vector<Work> reduce;
      std::vector<double> cost;
      int64_t slots = 0;
      for (int i = 0; i < n; ++i) {
        const int ks = stages(w[i]), want = i < whole ? 1 : (int)std::min(32.0, std::ceil(ks / limit));
        const int per = ns_part(ks, want, accurate), parts = (ks + per - 1) / per;
        if (parts <= 1) {
          items.push_back({w[i], (double)ks});
        } else {
          reduce.push_back(Work{w[i].mat, w[i].a, w[i].b | parts, (int)slots});
          for (int p = 0; p < parts; ++p, ++slots)
            items.push_back({Work{w[i].mat, w[i].a | p, w[i].b | parts, (int)slots}, (double)std::min(per, ks - p * per)});
        }
      }
      const double stage = tc.stage + (tc.full - tc.stage) * std::min(1.0, (double)items.size() / kCus);
      for (Item& x : items) cost.push_back(x.cost = x.cost * stage + fixed);
      double time = std::max(makespan(cost), total * tc.full / kCus);
      if (slots) time += kLaunch + (2.0 * slots + reduce.size()) * tile_bytes / kMemory;
      // a split has to promise a twentieth: the model is no better than that
      if (best.tile && time >= (slots ? 0.95 : 1.0) * best.time) return;
      best.tile = tc.tile;
      best.time = time;
      best.slots = slots;
      best.work = spread(items);
      best.reduce = reduce;
      while (best.reduce.size() % kXcds) best.reduce.push_back(Work{-1, 0, 0, 0});
    };
    consider(1.0, n);
    if (st == NS_UPDATE || n > 8 * kCus) continue;
    for (double share : {1.0, 0.75, 0.5, 0.34, 0.25}) {      // of a CU's share of the list
      const double limit = std::max(4.0, share * total / kCus);
      consider(limit, 0);
      if (n > kCus) consider(limit, n / kCus * kCus);
    }
  }
  return best;
}

}  // namespace

NsGroup::~NsGroup() { if (buf_) (void)hipFree(buf_); }

hipError_t NsGroup::create(const std::vector<Item>& items, int in_type, int out_type, bool accurate) {
  it_ = in_type;
  ot_ = out_type;
  accurate_ = accurate;
  const int n = (int)items.size();
  // A group whose X, A and B exceed the card, padded to the narrowest tiles, is refused before its tiles
  // are listed: 2^22 x 2^22 has 2^32 of them. What passes has 10^7 at most.
  size_t card_free = 0, card = 0;
  hipError_t e = hipMemGetInfo(&card_free, &card);
  if (e != hipSuccess) return e;
  for (const Item& t : items) {
    const size_t s = (size_t)rup(std::min(t.m, t.n), 64), l = (size_t)rup(std::max(t.m, t.n), 64);
    bytes_ += 8 * s * l + (accurate ? 8 : 4) * s * s;
    if (bytes_ > card) return hipErrorOutOfMemory;
  }
  std::vector<NsMat> mats(n);
  struct Off { size_t xh[2], xl[2], ah, al, bh, bl, partial; };
  std::vector<Off> offs(n);
  size_t ws = 0;
  auto take = [&](size_t bytes) { const size_t o = ws; ws += (bytes + 255) / 256 * 256; return o; };
  for (int i = 0; i < n; ++i) {
    const Item& t = items[i];
    NsMat& d = mats[i];
    std::memset(&d, 0, sizeof d);
    d.in = t.in; d.ld_in = t.ld_in; d.mom = t.mom; d.out = t.out; d.ld_out = t.ld_out;
    d.m = (int)t.m; d.n = (int)t.n;
    d.flip = t.m > t.n;
    d.s = std::min(d.m, d.n); d.l = std::max(d.m, d.n);
    // parts of at least 4096 elements, at most 1024 of them (every X0 workgroup adds them up)
    d.part_rows = (int)std::max<int64_t>((4096 + t.n - 1) / t.n, (t.m + 1023) / 1024);
    d.parts = (d.m + d.part_rows - 1) / d.part_rows;
  }
  const Planned plan[3] = {plan_list(mats, NS_GRAM, accurate), plan_list(mats, NS_POLY, accurate),
                           plan_list(mats, NS_UPDATE, accurate)};
  const int square = std::max(plan[0].tile, plan[1].tile), pad_s = std::max(square, plan[2].tile);
  const int64_t slots = std::max(plan[0].slots * plan[0].tile * plan[0].tile, plan[1].slots * plan[1].tile * plan[1].tile);
  for (int i = 0; i < n; ++i) {
    NsMat& d = mats[i];
    d.sp = (int)rup(d.s, pad_s);
    d.lp = (int)rup(d.l, plan[2].tile);
    const size_t x = (size_t)d.sp * d.lp * 2, a = (size_t)d.sp * d.sp * 2;
    Off& o = offs[i];
    for (int k = 0; k < 2; ++k) { o.xh[k] = take(x); o.xl[k] = take(x); }
    o.ah = take(a);
    o.bh = take(a);
    o.al = accurate ? take(a) : 0;
    o.bl = accurate ? take(a) : 0;
    o.partial = take((size_t)d.parts * 8);
  }
  const size_t slots_off = take((size_t)slots * 4);

  std::vector<Work> all;
  auto add = [&](List& l, const std::vector<Work>& w) {
    l.off = (int)all.size();
    l.cnt = (int)w.size();
    all.insert(all.end(), w.begin(), w.end());
  };
  std::vector<Work> w;
  for (int i = 0; i < n; ++i)
    for (int p = 0; p < mats[i].parts; ++p) w.push_back(Work{i, p * mats[i].part_rows, p, 0});
  add(norm_, w);
  w.clear();
  const int xt = ns_x0_tile();
  for (int i = 0; i < n; ++i)
    for (int a = 0; a < mats[i].sp; a += xt)
      for (int b = 0; b < mats[i].lp; b += xt) w.push_back(Work{i, a, b, 0});
  add(x0_, w);
  size_t n_items = 0;
  for (const Planned& p : plan) n_items += p.work.size() + p.reduce.size();
  const size_t mats_off = take(sizeof(NsMat) * n), work_off = take(sizeof(Work) * all.size()), zero_off = take(sizeof(int32_t)),
               items_off = take(sizeof(NsItem) * n_items);
  bytes_ = ws;
  e = device_alloc(&buf_, bytes_);
  if (e != hipSuccess) return hipErrorOutOfMemory;
  char* base = static_cast<char*>(buf_);
  d_mats_ = reinterpret_cast<NsMat*>(base + mats_off);
  d_work_ = reinterpret_cast<Work*>(base + work_off);
  d_zero_ = reinterpret_cast<int32_t*>(base + zero_off);
  for (int i = 0; i < n; ++i) {
    NsMat& d = mats[i];
    const Off& o = offs[i];
    for (int k = 0; k < 2; ++k) {
      d.xh[k] = reinterpret_cast<uint16_t*>(base + o.xh[k]);
      d.xl[k] = reinterpret_cast<uint16_t*>(base + o.xl[k]);
    }
    d.ah = reinterpret_cast<uint16_t*>(base + o.ah);
    d.bh = reinterpret_cast<uint16_t*>(base + o.bh);
    d.al = accurate ? reinterpret_cast<uint16_t*>(base + o.al) : nullptr;
    d.bl = accurate ? reinterpret_cast<uint16_t*>(base + o.bl) : nullptr;
    d.partial = reinterpret_cast<double*>(base + o.partial);
    d.factor[0] = (float)std::sqrt(std::max(1.0, (double)d.m / d.n));
    d.factor[1] = (float)(0.2 * std::sqrt((double)std::max(d.m, d.n)));
  }
  std::vector<NsItem> items_h;
  items_h.reserve(n_items);
  NsItem* const d_items = reinterpret_cast<NsItem*>(base + items_off);
  auto put = [&](const std::vector<Work>& list) {
    const NsItem* at = d_items + items_h.size();
    for (const Work& x : list) items_h.push_back(NsItem{x, mats[std::max(x.mat, 0)]});
    return at;
  };
  NsList* const out[3] = {&gram_, &poly_, &update_};
  for (int k = 0; k < 3; ++k) {
    out[k]->tile = plan[k].tile;
    out[k]->work = put(plan[k].work);
    out[k]->n_work = (int)plan[k].work.size();
    out[k]->reduce = put(plan[k].reduce);
    out[k]->n_reduce = (int)plan[k].reduce.size();
    out[k]->partial = reinterpret_cast<float*>(base + slots_off);
  }
  const int32_t zero = 0;
  if ((e = hipMemcpy(d_mats_, mats.data(), sizeof(NsMat) * n, hipMemcpyHostToDevice)) != hipSuccess) return e;
  if ((e = hipMemcpy(d_work_, all.data(), sizeof(Work) * all.size(), hipMemcpyHostToDevice)) != hipSuccess) return e;
  if ((e = hipMemcpy(d_zero_, &zero, sizeof zero, hipMemcpyHostToDevice)) != hipSuccess) return e;
  if ((e = hipMemcpy(d_items, items_h.data(), sizeof(NsItem) * n_items, hipMemcpyHostToDevice)) != hipSuccess) return e;
  return hipDeviceSynchronize();
}

hipError_t NsGroup::run(const NsArgs& args, int adjust, hipStream_t s) {
  NsArgs a = args;
  a.adjust = adjust;
  if (!a.skip) a.skip = d_zero_;
  auto W = [&](const List& l) { return d_work_ + l.off; };
  hipError_t e = launch_ns_norm(it_, d_mats_, W(norm_), norm_.cnt, a, s);
  if (e == hipSuccess) e = launch_ns_x0(it_, d_mats_, W(x0_), x0_.cnt, a, s);
  for (int k = 0; k < a.steps && e == hipSuccess; ++k) {
    e = launch_ns_gemm(NS_GRAM, accurate_, ot_, false, gram_, k, a, s);
    if (e == hipSuccess) e = launch_ns_gemm(NS_POLY, accurate_, ot_, false, poly_, k, a, s);
    if (e == hipSuccess) e = launch_ns_gemm(NS_UPDATE, accurate_, ot_, k + 1 == a.steps, update_, k, a, s);
  }
  return e;
}

}  // namespace psgd
