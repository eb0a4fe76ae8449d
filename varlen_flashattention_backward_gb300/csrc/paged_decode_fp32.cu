// fa_paged_decode, fp32.

#include "paged_decode.cuh"

namespace fav {

namespace {

template <int D>
int warps_simt(int rows) {
  return rows == 1   ? SimtShape<D, 1>::NT
         : rows == 2 ? SimtShape<D, 2>::NT
         : rows == 4 ? SimtShape<D, 4>::NT
                     : SimtShape<D, 8>::NT;
}

template <int D>
int teams_of_d(bool tc, int rows) {
  if (!tc) return warps_simt<D>(rows);
  return rows == 8    ? TcShape<D, 8>::NT
         : rows == 16 ? TcShape<D, 16>::NT
         : rows == 32 ? TcShape<D, 32>::NT
                      : TcShape<D, 64>::NT;
}

int teams_of(bool tc, int rows, int d) {
  switch (d) {
    case 32: return teams_of_d<32>(tc, rows);
    case 64: return teams_of_d<64>(tc, rows);
    case 96: return teams_of_d<96>(tc, rows);
    case 128: return teams_of_d<128>(tc, rows);
    default: return teams_of_d<192>(tc, rows);
  }
}

}  // namespace

// The shape of a call, from its scalars alone.
DecodePlan decode_plan(fa_dtype dt, int batch, int n_kv, int group, int d, int64_t max_keys,
                       int sms) {
  DecodePlan plan;
  // fp32: the heads whose outputs a lane's registers hold at once.  16-bit types:
  // 8 rows per warp, whose products serve P twice, or 16, or teams of warps with
  // 16 each; larger groups are cut, and read their keys again.
  const bool tc = dt != FA_DTYPE_FP32;
  if (tc)
    plan.rows = group <= 8 ? 8 : group <= 16 ? 16 : group <= 32 ? 32 : 64;
  else
    plan.rows = group <= 1 ? 1 : group <= 2 ? 2 : group <= 4 ? 4 : 8;
  plan.teams = teams_of(tc, plan.rows, d);
  // The largest cluster per segment that still puts all of them on the GPU at
  // once, if its teams get at most kDirectBlocks blocks each.  Clusters share a
  // GPC, so fewer large ones fit than SMs would hold (152 SMs: 15 of eight, 36 of
  // four, 76 of two); a second wave doubles the time.  Of single CTAs, two waves: on the
  // GPU they take 1.6 us less than ranges and a join to 1.8 us more (61 requests of up to
  // 128 keys, 4 key heads 8.8 us and 10.4; 32 of up to 512, 8 key heads 13.8 and 12.0; 32
  // of 512 16.3 and 15.2), but the host saves a launch and a workspace: calls on a stream
  // take 8.6 and 18.6, 13.7 and 18.3, 16.2 and 19.2 us.
  const int kb = tc ? 16 : 8;
  const int64_t blocks = (max_keys + kb - 1) / kb + 1;
  const int64_t segments = int64_t(batch) * n_kv * ((group + plan.rows - 1) / plan.rows);
  const auto fits = [&](int ctas) {
    const int percent = ctas == 1 ? 200 : ctas == 2 ? 95 : ctas == 4 ? 85 : 63;
    return segments * ctas * 100 <= int64_t(sms) * percent;
  };
  int ctas = 1;
  while (ctas < kMaxDirect && fits(ctas * 2) && ctas * plan.teams < blocks) ctas *= 2;
  plan.direct =
      fits(ctas) && blocks <= int64_t(ctas) * plan.teams * kDirectBlocks ? ctas : 0;
  return plan;
}

size_t decode_part_floats(int rows, int d) { return size_t(slot_floats(rows, d)); }

cudaError_t launch_paged_decode_fp32(const DecodeParams &p, int sms, cudaStream_t s) {
  FAV_DECODE_BY_DIM(launch_simt, );
}

}  // namespace fav
