// Host side of the Newton-Schulz group: layout, tile lists, and the launches of one call.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <cstdlib>

#include "ns.h"

namespace psgd {
int ns_x0_tile();

namespace {

inline int64_t rup(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// Spread a tile list over the XCDs (xcd_remap: XCD x walks the x-th eighth of the list). Groups
// of `gsize` consecutive items share an operand panel and stay on one XCD, longest group first
// to the XCD with the least work so far; short lists are dealt out item by item, since a shared
// panel is worth less than an idle XCD.
void balance(std::vector<Work>& w, std::vector<int64_t>& cost, const std::vector<int>& group) {
  const int n = (int)w.size();
  const bool single = n <= 512;
  struct G { int beg, end; int64_t c; };
  std::vector<G> gs;
  for (int i = 0; i < n;) {
    int j = i;
    int64_t c = 0;
    while (j < n && (single ? j == i : group[j] == group[i])) c += cost[j++];
    gs.push_back({i, j, c});
    i = j;
  }
  std::stable_sort(gs.begin(), gs.end(), [](const G& a, const G& b) { return a.c > b.c; });
  std::vector<std::vector<Work>> seg(kXcds);
  int64_t load[kXcds] = {};
  for (const G& g : gs) {
    int x = 0;
    for (int y = 1; y < kXcds; ++y) if (load[y] < load[x]) x = y;
    load[x] += g.c;
    for (int i = g.beg; i < g.end; ++i) seg[x].push_back(w[i]);
  }
  size_t per = 0;
  for (const auto& s : seg) per = std::max(per, s.size());
  w.clear();
  for (auto& s : seg) {
    s.resize(per, Work{-1, 0, 0, 0});
    w.insert(w.end(), s.begin(), s.end());
  }
}

}  // namespace

NsGroup::~NsGroup() { if (buf_) (void)hipFree(buf_); }

hipError_t NsGroup::create(const std::vector<Item>& items, int in_type, int out_type, bool accurate) {
  it_ = in_type;
  ot_ = out_type;
  accurate_ = accurate;
  const int n = (int)items.size();
  // 128-wide tiles reuse each staged value twice as often; 64-wide ones fill the chip when the
  // group is small
  int64_t tiles = 0;
  for (const Item& t : items)
    tiles += (rup(std::min(t.m, t.n), 128) / 128) * (rup(std::max(t.m, t.n), 128) / 128);
  tile_ = tiles >= 256 ? 128 : 64;
  if (getenv("NS_TILE")) tile_ = atoi(getenv("NS_TILE"));

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
    d.sp = (int)rup(d.s, tile_); d.lp = (int)rup(d.l, tile_);
    // parts of at least 8192 elements, at most 1024 of them (every X0 workgroup adds them up)
    d.part_rows = (int)std::max<int64_t>((8192 + t.n - 1) / t.n, (t.m + 1023) / 1024);
    d.parts = (d.m + d.part_rows - 1) / d.part_rows;
    const size_t x = (size_t)d.sp * d.lp * 2, a = (size_t)d.sp * d.sp * 2;
    Off& o = offs[i];
    for (int k = 0; k < 2; ++k) { o.xh[k] = take(x); o.xl[k] = take(x); }
    o.ah = take(a);
    o.bh = take(a);
    o.al = accurate ? take(a) : 0;
    o.bl = accurate ? take(a) : 0;
    o.partial = take((size_t)d.parts * 8);
  }

  std::vector<Work> all;
  auto add = [&](List& l, const std::vector<Work>& w) {
    l.off = (int)all.size();
    l.cnt = (int)w.size();
    all.insert(all.end(), w.begin(), w.end());
  };
  std::vector<Work> w;
  std::vector<int64_t> cost;
  std::vector<int> group;
  auto clear = [&] { w.clear(); cost.clear(); group.clear(); };
  for (int i = 0; i < n; ++i)
    for (int p = 0; p < mats[i].parts; ++p) w.push_back(Work{i, p * mats[i].part_rows, p, 0});
  add(norm_, w);
  clear();
  const int xt = ns_x0_tile();
  for (int i = 0; i < n; ++i)
    for (int a = 0; a < mats[i].sp; a += xt)
      for (int b = 0; b < mats[i].lp; b += xt) w.push_back(Work{i, a, b, 0});
  add(x0_, w);
  int gid = 0;
  for (int st = 0; st < 2; ++st) {         // A, then B: tiles on and below the diagonal
    clear();
    for (int i = 0; i < n; ++i)
      for (int a = 0; a < mats[i].sp; a += tile_, ++gid)
        for (int b = 0; b <= a; b += tile_) {
          w.push_back(Work{i, a, b, 0});
          cost.push_back(st == 0 ? mats[i].l : mats[i].s);
          group.push_back(gid);
        }
    balance(w, cost, group);
    add(st == 0 ? gram_ : poly_, w);
  }
  clear();
  for (int i = 0; i < n; ++i)              // X: the row tiles over one column panel share it
    for (int a = 0; a < mats[i].lp; a += tile_, ++gid)
      for (int b = 0; b < mats[i].sp; b += tile_) {
        w.push_back(Work{i, a, b, 0});
        cost.push_back(mats[i].s);
        group.push_back(gid);
      }
  balance(w, cost, group);
  add(update_, w);

  const size_t mat_bytes = (sizeof(NsMat) * n + 255) / 256 * 256;
  const size_t work_off = ws + 2 * mat_bytes;
  bytes_ = work_off + sizeof(Work) * all.size();
  hipError_t e = hipMalloc(&buf_, bytes_);
  if (e != hipSuccess) { buf_ = nullptr; return hipErrorOutOfMemory; }
  char* base = static_cast<char*>(buf_);
  d_work_ = reinterpret_cast<Work*>(base + work_off);
  for (int adj = 0; adj < 2; ++adj) {
    d_mats_[adj] = reinterpret_cast<NsMat*>(base + ws + adj * mat_bytes);
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
      d.factor = adj == 0 ? (float)std::sqrt(std::max(1.0, (double)d.m / d.n))
                          : (float)(0.2 * std::sqrt((double)std::max(d.m, d.n)));
    }
    if ((e = hipMemcpy(d_mats_[adj], mats.data(), sizeof(NsMat) * n, hipMemcpyHostToDevice)) != hipSuccess) return e;
  }
  if ((e = hipMemcpy(d_work_, all.data(), sizeof(Work) * all.size(), hipMemcpyHostToDevice)) != hipSuccess) return e;
  return hipDeviceSynchronize();
}

hipError_t NsGroup::run(const NsArgs& a, int adjust, hipStream_t s) {
  const NsMat* dm = d_mats_[adjust];
  auto W = [&](const List& l) { return d_work_ + l.off; };
  hipError_t e = launch_ns_norm(it_, dm, W(norm_), norm_.cnt, a, s);
  if (e == hipSuccess) e = launch_ns_x0(it_, dm, W(x0_), x0_.cnt, a, s);
  for (int k = 0; k < a.steps && e == hipSuccess; ++k) {
    e = launch_ns_gemm(NS_GRAM, tile_, accurate_, ot_, false, dm, W(gram_), gram_.cnt, k, a, s);
    if (e == hipSuccess) e = launch_ns_gemm(NS_POLY, tile_, accurate_, ot_, false, dm, W(poly_), poly_.cnt, k, a, s);
    if (e == hipSuccess) e = launch_ns_gemm(NS_UPDATE, tile_, accurate_, ot_, k + 1 == a.steps, dm, W(update_), update_.cnt, k, a, s);
  }
  return e;
}

}  // namespace psgd
