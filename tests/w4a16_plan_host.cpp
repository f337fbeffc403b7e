// The whole-number functions of csrc/w4a16_plan.hpp for tests/test_w4a16_plan.py: a wave's lanes one after the other.
#include "w4a16_plan.hpp"

using namespace mxf;

namespace {

template <int BM, int CE>
bool item_of(const int32_t* off, int E, int64_t R, int lo, int hi, int ntiles, int x, int j, int64_t* out) {
  int o[64][CE + 1], units[64], total = 0;
  for (int lane = 0; lane < 64; ++lane) total += units[lane] = w16_lane_units<BM, CE>(off, E, R, lo, hi, lane, o[lane]);
  uint32_t w;
  if (!w16_range((uint32_t)total * (uint32_t)ntiles, x, j, w)) return false;
  const int p = (int)(w / (uint32_t)ntiles);
  int before = 0, lane = 0;
  while (lane < 64 && !(p >= before && p < before + units[lane])) before += units[lane++];
  if (lane == 64) return false;
  const W16Pick k = w16_lane_find<BM, CE>(off, E, R, lo, hi, lane, o[lane], before, p);
  int n, m;
  int64_t row0;
  if (!w16_item_place<BM>(k, w, ntiles, n, row0, m)) return false;
  out[0] = k.e, out[1] = n, out[2] = row0, out[3] = m;
  return true;
}

template <int BM>
bool item(const int32_t* off, int E, int64_t R, int lo, int hi, int ntiles, int x, int j, int64_t* out) {
  if (E <= 64) return item_of<BM, 1>(off, E, R, lo, hi, ntiles, x, j, out);
  if (E <= 256) return item_of<BM, 4>(off, E, R, lo, hi, ntiles, x, j, out);
  return item_of<BM, 0>(off, E, R, lo, hi, ntiles, x, j, out);
}

}  // namespace

extern "C" {

// the items (expert, n-tile, first row, rows) that the workgroups of a launch take; returns how many
int64_t items(int bm, const int32_t* off, int E, int64_t R, int lo, int hi, int64_t ntiles, int64_t workgroups, int64_t* out) {
  int64_t n = 0;
  for (int64_t b = 0; b < workgroups; ++b) {
    const int x = (int)(b & 7), j = (int)(b >> 3);
    const bool ok = bm == 16   ? item<16>(off, E, R, lo, hi, (int)ntiles, x, j, out + 4 * n)
                    : bm == 64 ? item<64>(off, E, R, lo, hi, (int)ntiles, x, j, out + 4 * n)
                               : item<128>(off, E, R, lo, hi, (int)ntiles, x, j, out + 4 * n);
    n += ok;
  }
  return n;
}

// the same of one matrix: (unit, n-tile)
int64_t matrix_items(int64_t units, int64_t ntiles, int64_t workgroups, int64_t* out) {
  int64_t n = 0;
  for (int64_t b = 0; b < workgroups; ++b) {
    uint32_t w;
    if (!w16_range((uint32_t)(units * ntiles), (int)(b & 7), (int)(b >> 3), w)) continue;
    int t, u;
    w16_place(w, (uint32_t)units, (uint32_t)ntiles, t, u);
    out[2 * n] = u, out[2 * n + 1] = t;
    ++n;
  }
  return n;
}

int grouped_plan(int64_t R, int E, int64_t N, int64_t K, int nv, int swiglu, int64_t* out) {
  W16Launch l[3];
  const int n = w16_grouped_plan(R, E, N, K, nv != 0, swiglu != 0, l);
  for (int i = 0; i < n; ++i) {
    const int64_t v[6] = {l[i].bm, l[i].bn, l[i].min_rows, l[i].max_rows, l[i].workgroups(), l[i].ntiles};
    for (int j = 0; j < 6; ++j) out[6 * i + j] = v[j];
  }
  return n;
}

int segment(const int32_t* seg_off, int S, int64_t t) {
  int lo = 0, hi = S;
  while (lo < hi) {
    const bool one = w16_probe_step(lo, hi) == 1;
    unsigned long long mask = 0;
    for (int lane = 0; lane < 64; ++lane) mask |= (unsigned long long)w16_probe(seg_off, lo, hi, lane, t) << lane;
    w16_probe_narrow(mask, lo, hi);
    if (one) break;
  }
  return lo;
}

uint32_t share(uint32_t n, int i, int s) { return w16_share(n, i, s); }
int swizzle_a(int r) { return swz_a16(r); }
int swizzle_b(int r) { return swz_b16(r); }
int64_t weight_row(int swiglu, int BN, int64_t half, int n, int r) { return w16_weight_row(swiglu != 0, BN, half, n, r); }
int issues_codes(int i, int st, int nst) { return w16_issues_codes(i, st, nst); }
int begins_scales(int st, int st0, int P, int nst) { return w16_begins_scales(st, st0, P, nst); }
int issues_a(int st, int NA, int nst) { return w16_issues_a(st, NA, nst); }
int a_slot(int i, int NA) { return w16_a_slot(i, NA); }
int code_slot(int i) { return w16_code_slot(i); }
int turn(int NA) { return w16_turn(NA); }
int in_flight(int i, int NA, int IA, int IB, int last, int scales) { return w16_in_flight(i, NA, IA, IB, last, scales); }
}
