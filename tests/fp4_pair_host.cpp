// The whole-number functions of csrc/fp4_pair_plan.hpp for tests/test_fp4_pair_replay.py: one operand's copies and
// reads, all chunks, lanes or rows after each other.
#include "fp4_pair_plan.hpp"

using namespace mxf;

extern "C" {

void plan(int64_t M, int64_t N, int64_t K, int nv, int32_t* out) {
  const Fp4PairPlan p = fp4_pair_plan(M, N, K, nv != 0);
  out[0] = p.bm, out[1] = p.bn, out[2] = p.slices;
}

uint32_t share(uint32_t n, int i, int s) { return w16_share(n, i, s); }
int group_stages(int nv) { return pair_group_stages(nv != 0); }
int begins_scales(int st, int st0, int nv, int nst) { return w16_begins_scales(st, st0, pair_group_stages(nv != 0), nst); }
int past(int g, int st, int64_t K) { return pair_past(g, st, K); }
int few_copies() { return kFewCopies; }
int few_loads() { return kFewLoads; }

// the source of 16-byte copy c of a slot, for each of them
void copies(int rows, int64_t wrow, int64_t* out) {
  for (int c = 0; c < rows * 8; ++c) out[c] = pair_copy_from(c, wrow);
}
// the source of the 16 bytes that part p's lane l copies, at 64 p + l
void scales(int rows, int64_t srow, int64_t* out) {
  for (int i = 0; i < rows * 2; ++i) out[i] = pair_scales_from(i / 64, i % 64, srow);
}
// where a lane of group g reads step s of row r: [rows][2][4]
void blocks(int rows, int32_t* out) {
  for (int r = 0; r < rows; ++r)
    for (int g = 0; g < 2; ++g)
      for (int s = 0; s < 4; ++s) *out++ = pair_step(pair_block_at(r, g), s);
}
// where it finds its scales of a stage: [rows][2]
void scales_at(int rows, int st, int nv, int32_t* out) {
  for (int r = 0; r < rows; ++r)
    for (int g = 0; g < 2; ++g) *out++ = pair_scales_at(st, g, nv != 0) + pair_scales_row(r);
}
// the few-tile kernel's loads of scales: [32][2]
void few_scales(int st, int64_t srow, int nv, int64_t* out) {
  for (int r = 0; r < 32; ++r)
    for (int g = 0; g < 2; ++g) *out++ = (int64_t)pair_few_scales(r, g, srow, nv != 0) + pair_few_scales_step(st, nv != 0);
}
int out_to(int f, int j, int g, int r, int es, int chunks) { return pair_out_to(f, j, g, r, es, chunks); }
int out_from(int r, int c, int chunks) { return pair_out_from(r, c, chunks); }
int few_sum(int r, int c) { return pair_few_sum(r, c); }

}
