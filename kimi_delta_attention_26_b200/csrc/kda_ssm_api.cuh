// kda_ssm_api.cuh -- argument checks and launches of the scan's entry points.
// Part of kda_api.cu's translation unit, after kda_conv_api.cuh.
#pragma once

namespace {

constexpr int64_t kSsmMaxChannels = 1 << 17;
constexpr int64_t kSsmMaxStates = 128;

struct SsmArgs {
  int64_t T, C, N, G;
  kda_dtype_t dt;
  RowView u, dt_, b, c, z, out;  // out: dout for the backward pass
  void *A, *D, *bias;
  Span s_A, s_D, s_bias;
};

kda_status_t check_ssm(const kda_tensor_t* u, const kda_tensor_t* dt, const kda_tensor_t* A, const kda_tensor_t* B,
                       const kda_tensor_t* C, const kda_tensor_t* D, const kda_tensor_t* z, const kda_tensor_t* dt_bias,
                       const kda_tensor_t* out, bool written, SsmArgs* a) {
  if (!u || !dt || !A || !B || !C || !out) return KDA_ERR_NULL;
  if (!io_bytes(u->dtype)) return KDA_ERR_DTYPE;
  if (u->ndim != 2 || A->ndim != 2 || B->ndim != 3) return KDA_ERR_SHAPE;
  a->dt = u->dtype;
  a->T = u->shape[0];
  a->C = u->shape[1];
  a->N = A->shape[1];
  a->G = B->shape[1];
  if (a->T < 0 || a->T > kMaxRows || a->C < 1 || a->C > kSsmMaxChannels || a->N < 1 || a->N > kSsmMaxStates ||
      a->G < 1 || a->G > a->C || a->C % a->G != 0)
    return KDA_ERR_SHAPE;
  kda_status_t st;
  if ((st = view_rows(u, a->dt, a->T, 0, a->C, false, &a->u)) != KDA_OK ||
      (st = view_rows(dt, a->dt, a->T, 0, a->C, false, &a->dt_)) != KDA_OK ||
      (st = view_packed(A, KDA_F32, {a->C, a->N}, false, &a->A, &a->s_A)) != KDA_OK ||
      (st = view_rows(B, a->dt, a->T, a->G, a->N, false, &a->b)) != KDA_OK ||
      (st = view_rows(C, a->dt, a->T, a->G, a->N, false, &a->c)) != KDA_OK ||
      (st = view_packed(D, KDA_F32, {a->C}, true, &a->D, &a->s_D)) != KDA_OK ||
      (z && (st = view_rows(z, a->dt, a->T, 0, a->C, false, &a->z)) != KDA_OK) ||
      (st = view_packed(dt_bias, KDA_F32, {a->C}, true, &a->bias, &a->s_bias)) != KDA_OK ||
      (st = view_rows(out, a->dt, a->T, 0, a->C, written, &a->out)) != KDA_OK)
    return st;
  return KDA_OK;
}

// The time split: tokens per range (a multiple of 16), or 0. A range's blocks run
// beside the other ranges'; first passes over the pieces that cross a border
// give each range's start (and, for the gradients, its end).
//
// Ranges are chosen to fill the places that the device has for blocks once, twice
// or three times, by the time that a block's chain of tokens takes: rounds x (a
// range's tokens + a start), times what the first passes add (`alone`), and
// more where blocks share an SM (`shared`). The split is taken where that is a
// tenth less than the longest sequence's chain. The lengths are on the device, so
// several sequences' longest is taken to be 5/4 of the mean.
// Measured, us (one sequence unless stated; bf16), the split as the rule takes it:
//                                   forward          gradients
//                                split  unsplit    split  unsplit
//   32768 x 1024 x 16 states       444     1112     1435    10512
//   8192 x 2048 x 16               231      286      742     2685
//   2048 x 1024 x 16                49       78      157      648
//   512 x 1024 x 16                                   81      185
//   1000 + 1000, 1024 x 16                           144      334
//   1024 x 4096 x 16                                 232      367
// and by force where the rule leaves it:
//   1024 x 2048 x 16                48       43
//   1000 + 1000, 1024 x 16          45       43
//   8 of 512 tokens, 256 x 16       41       26
//   4 of 256 tokens, 2048 x 16                       133      114
//   8 of 512 tokens, 512 x 24                        275      224
//   4 of 4096 tokens, 1024 x 24                     2013     1593
// Where it is wrong, one long sequence among short ones:
//   32000 + 7 of 110, 1024 x 16    448     1259     1458    10377  (the gradients do split)
//   32000 + 15 of 50, 1024 x 16                     1477    10283
//   8192 + 1 + 1, 4096 x 16        421      533     1382     2831
struct SplitCost {
  int resident;   // blocks that an SM holds
  int64_t least;  // tokens of a range, at least
  // in tokens' time of a block that is alone on its SM:
  int start;      // a block's start
  int launches;   // the first passes' launches
  float alone, shared;
};

int64_t split_run(const SsmArgs& a, int32_t num_seqs, int64_t blocks, const SplitCost& c, int dev) {
  const int mode = g_split.load();
  if (mode == 1) return 0;
  if (mode == 2) return a.T >= 128 ? std::max<int64_t>(64, (a.T / 65535 + 32) / 32 * 32) : 0;  // testing
  const int64_t sms = g_num_sms[dev], places = c.resident * sms;
  if (blocks * num_seqs > sms) return 0;
  int64_t best = 0;
  const int64_t longest = num_seqs == 1 ? a.T : a.T * 5 / (4 * static_cast<int64_t>(num_seqs));
  float best_cost = 0.9f * (longest + c.start);
  for (int rounds = 1; rounds <= 3; ++rounds) {
    int64_t ranges = std::min<int64_t>(rounds * places / blocks, a.T / c.least);
    if (ranges < 2) continue;
    const int64_t run = ((a.T + ranges - 1) / ranges + 15) / 16 * 16;
    ranges = (a.T + run - 1) / run;
    const float cost = ((ranges * blocks + places - 1) / places) * (run + c.start) *
                           (ranges * blocks > sms && c.resident > 1 ? c.shared : c.alone) + c.launches;
    if (cost < best_cost) best = run, best_cost = cost;
  }
  return best;
}

int64_t scan_blocks(const SsmArgs& a) {
  const int ch = kda::ssm::scan_channels(static_cast<int>(a.N));
  return a.G * ((a.C / a.G + ch - 1) / ch);
}

kda::ssm::Params ssm_params(const SsmArgs& a, int32_t softplus, const int32_t* cu, int32_t num_seqs, const void* init) {
  kda::ssm::Params p;
  std::memset(&p, 0, sizeof(p));
  p.u = a.u.data;
  p.dt = a.dt_.data;
  p.z = a.z.data;
  p.b = a.b.data;
  p.c = a.c.data;
  p.A = static_cast<const float*>(a.A);
  p.D = static_cast<const float*>(a.D);
  p.dt_bias = static_cast<const float*>(a.bias);
  p.cu = cu;
  p.init = static_cast<const float*>(init);
  p.T = a.T;
  p.u_st = a.u.st;
  p.dt_st = a.dt_.st;
  p.z_st = a.z.st;
  p.b_st = a.b.st;
  p.b_sg = a.b.sg;
  p.c_st = a.c.st;
  p.c_sg = a.c.sg;
  p.NS = num_seqs;
  p.C = static_cast<int>(a.C);
  p.N = static_cast<int>(a.N);
  p.G = static_cast<int>(a.G);
  p.softplus = softplus;
  // two channels at a time: every block's and group's first channel is even
  const int pair = 2 * io_bytes(a.dt), quad = 2 * pair;
  const bool even = a.C / a.G % 2 == 0 || a.G == 1;
  p.wide = (even && aligned(a.u, pair) ? 1 : 0) | (even && aligned(a.dt_, pair) ? 2 : 0) | (even && aligned(a.z, pair) ? 4 : 0) |
           (a.N % 4 == 0 && aligned(a.b, quad) ? 8 : 0) | (a.N % 4 == 0 && aligned(a.c, quad) ? 16 : 0) |
           (even && aligned(a.out, pair) ? 32 : 0);
  return p;
}

}  // namespace

extern "C" {

kda_status_t kda_ssm_fwd(const kda_tensor_t* u, const kda_tensor_t* dt, const kda_tensor_t* A, const kda_tensor_t* B,
                         const kda_tensor_t* C, const kda_tensor_t* D, const kda_tensor_t* z,
                         const kda_tensor_t* dt_bias, int32_t dt_softplus, const int32_t* cu_seqlens, int32_t num_seqs,
                         const kda_tensor_t* initial_state, const kda_tensor_t* out, const kda_tensor_t* final_state,
                         void* stream) {
  namespace sm = kda::ssm;
  g_last_cuda_error[0] = '\0';
  SsmArgs a;
  kda_status_t st = check_ssm(u, dt, A, B, C, D, z, dt_bias, out, true, &a);
  if (st != KDA_OK) return st;
  if ((st = check_packing_args(cu_seqlens, num_seqs, a.T)) != KDA_OK) return st;
  void *init, *fin;
  Span s_init, s_fin;
  if ((st = view_packed(initial_state, KDA_F32, {num_seqs, a.C, a.N}, true, &init, &s_init)) != KDA_OK ||
      (st = view_packed(final_state, KDA_F32, {num_seqs, a.C, a.N}, true, &fin, &s_fin)) != KDA_OK)
    return st;
  // a block reads its part of the initial state before it writes that of the final one: they may be the same tensor
  if (any_overlap({a.out.span, s_fin},
                  {a.u.span, a.dt_.span, a.b.span, a.c.span, a.z.span, a.s_A, a.s_D, a.s_bias}) ||
      overlap(a.out.span, s_init) || (init != fin && overlap(s_fin, s_init)))
    return KDA_ERR_OVERLAP;
  int dev = 0;
  if ((st = prologue(&dev)) != KDA_OK) return st;
  sm::Params p = ssm_params(a, dt_softplus != 0, cu_seqlens, num_seqs, init);
  p.out = a.out.data;
  p.o_st = a.out.st;
  p.fin = static_cast<float*>(fin);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const int sms = g_num_sms[dev];
  const int64_t run = split_run(a, num_seqs, scan_blocks(a), {sm::scan_resident(static_cast<int>(a.N)), 192, 80, 300, 1.65f, 3.f}, dev);
  if (!run) {
    const cudaError_t e = by_type(a.dt, dev, [&](auto m) { return m.scan(p, sm::OUTPUTS, num_seqs, sms, cs); });
    return e != cudaSuccess ? cuda_fail(e) : KDA_OK;
  }
  if ((st = prepare_pool(dev)) != KDA_OK) return st;
  const int ranges = static_cast<int>((a.T + run - 1) / run);
  // A final state in the initial state's place is written behind the scan: its
  // last range's block may end before the first range's has read the state.
  const bool in_place = fin && fin == init;
  const size_t state_bytes = static_cast<size_t>(num_seqs) * a.C * a.N * 4;
  const size_t carry_bytes = round256(static_cast<size_t>(ranges) * a.C * a.N * 4);
  const size_t sum_bytes = round256(static_cast<size_t>(ranges) * a.C * 4);
  void* scratch = nullptr;
  cudaError_t e = pool_alloc(&scratch, carry_bytes + sum_bytes + (in_place ? state_bytes : 0), dev, cs);
  if (e != cudaSuccess) return cuda_fail(e);
  unsigned char* sb = static_cast<unsigned char*>(scratch);
  p.run = run;
  p.carry = reinterpret_cast<float*>(sb);
  p.sum_d = reinterpret_cast<float*>(sb + carry_bytes);
  if (in_place) p.fin = reinterpret_cast<float*>(sb + carry_bytes + sum_bytes);
  e = by_type(a.dt, dev, [&](auto m) {
    const cudaError_t f = ranges > 1 ? m.scan(p, sm::STATES, ranges - 1, sms, cs) : cudaSuccess;
    return f == cudaSuccess ? m.scan(p, sm::OUTPUTS, ranges, sms, cs) : f;
  });
  if (e == cudaSuccess && in_place) e = cudaMemcpyAsync(fin, p.fin, state_bytes, cudaMemcpyDeviceToDevice, cs);
  const cudaError_t ef = cudaFreeAsync(scratch, cs);
  if (e != cudaSuccess) return cuda_fail(e);
  return ef != cudaSuccess ? cuda_fail(ef) : KDA_OK;
}

kda_status_t kda_ssm_decode(const kda_tensor_t* u, const kda_tensor_t* dt, const kda_tensor_t* A, const kda_tensor_t* B,
                            const kda_tensor_t* C, const kda_tensor_t* D, const kda_tensor_t* z,
                            const kda_tensor_t* dt_bias, int32_t dt_softplus, const kda_tensor_t* state,
                            const int32_t* state_indices, const kda_tensor_t* out, void* stream) {
  namespace sm = kda::ssm;
  g_last_cuda_error[0] = '\0';
  SsmArgs a;
  kda_status_t st = check_ssm(u, dt, A, B, C, D, z, dt_bias, out, true, &a);
  if (st != KDA_OK) return st;
  if (!state) return KDA_ERR_NULL;
  if (state->ndim != 3) return KDA_ERR_SHAPE;
  const int64_t B_ = a.T, pool = state->shape[0];
  if (pool < 1 || (!state_indices && pool < B_) || pool > (int64_t(1) << 40) / (a.C * a.N)) return KDA_ERR_SHAPE;
  void* sp;
  Span s_state;
  if ((st = view_packed(state, KDA_F32, {pool, a.C, a.N}, false, &sp, &s_state)) != KDA_OK) return st;
  if (reinterpret_cast<uintptr_t>(state_indices) & 3u) return KDA_ERR_ALIGN;
  if (any_overlap({a.out.span, s_state},
                  {a.u.span, a.dt_.span, a.b.span, a.c.span, a.z.span, a.s_A, a.s_D, a.s_bias}))
    return KDA_ERR_OVERLAP;
  int dev = 0;
  if ((st = prologue(&dev)) != KDA_OK) return st;
  if (B_ == 0) return KDA_OK;
  sm::DecodeParams p;
  p.u = a.u.data;
  p.dt = a.dt_.data;
  p.z = a.z.data;
  p.b = a.b.data;
  p.c = a.c.data;
  p.A = static_cast<const float*>(a.A);
  p.D = static_cast<const float*>(a.D);
  p.dt_bias = static_cast<const float*>(a.bias);
  p.state = static_cast<float*>(sp);
  p.idx = state_indices;
  p.out = a.out.data;
  p.pool = pool;
  p.u_st = a.u.st;
  p.dt_st = a.dt_.st;
  p.z_st = a.z.st;
  p.o_st = a.out.st;
  p.b_st = a.b.st;
  p.b_sg = a.b.sg;
  p.c_st = a.c.st;
  p.c_sg = a.c.sg;
  p.C = static_cast<int>(a.C);
  p.N = static_cast<int>(a.N);
  p.G = static_cast<int>(a.G);
  p.softplus = dt_softplus != 0;
  const int quad = 4 * io_bytes(a.dt);
  p.wide = (a.N % 4 == 0 && aligned(a.b, quad) ? 1 : 0) | (a.N % 4 == 0 && aligned(a.c, quad) ? 2 : 0) |
           (a.N % 4 == 0 && aligned(sp, 16) && aligned(a.A, 16) ? 4 : 0) | (a.G > 1 && a.C / a.G % 4 != 0 ? 8 : 0);
  const cudaError_t e = by_type(a.dt, dev, [&](auto m) { return m.scan_decode(p, B_, static_cast<cudaStream_t>(stream)); });
  return e != cudaSuccess ? cuda_fail(e) : KDA_OK;
}

kda_status_t kda_ssm_bwd(const kda_tensor_t* u, const kda_tensor_t* dt, const kda_tensor_t* A, const kda_tensor_t* B,
                         const kda_tensor_t* C, const kda_tensor_t* D, const kda_tensor_t* z,
                         const kda_tensor_t* dt_bias, int32_t dt_softplus, const int32_t* cu_seqlens, int32_t num_seqs,
                         const kda_tensor_t* initial_state, const kda_tensor_t* dout, const kda_tensor_t* dfinal_state,
                         const kda_tensor_t* du, const kda_tensor_t* ddt, const kda_tensor_t* dA,
                         const kda_tensor_t* dB, const kda_tensor_t* dC, const kda_tensor_t* dD, const kda_tensor_t* dz,
                         const kda_tensor_t* ddt_bias, const kda_tensor_t* dinitial_state, void* stream) {
  namespace sm = kda::ssm;
  g_last_cuda_error[0] = '\0';
  SsmArgs a;
  kda_status_t st = check_ssm(u, dt, A, B, C, D, z, dt_bias, dout, false, &a);
  if (st != KDA_OK) return st;
  if ((st = check_packing_args(cu_seqlens, num_seqs, a.T)) != KDA_OK) return st;
  if ((z != nullptr) != (dz != nullptr)) return KDA_ERR_NULL;  // the gate and its gradient come together
  void *init, *dfin, *dinit, *da, *dd, *dbias;
  Span s_init, s_dfin, s_dinit, s_da, s_dd, s_dbias;
  RowView vdu, vddt, vdz, vdb, vdc;
  if ((st = view_packed(initial_state, KDA_F32, {num_seqs, a.C, a.N}, true, &init, &s_init)) != KDA_OK ||
      (st = view_packed(dfinal_state, KDA_F32, {num_seqs, a.C, a.N}, true, &dfin, &s_dfin)) != KDA_OK ||
      (st = view_rows(du, a.dt, a.T, 0, a.C, true, &vdu)) != KDA_OK ||
      (st = view_rows(ddt, a.dt, a.T, 0, a.C, true, &vddt)) != KDA_OK ||
      (st = view_packed(dA, KDA_F32, {a.C, a.N}, false, &da, &s_da)) != KDA_OK ||
      (st = view_rows(dB, a.dt, a.T, a.G, a.N, true, &vdb)) != KDA_OK ||
      (st = view_rows(dC, a.dt, a.T, a.G, a.N, true, &vdc)) != KDA_OK ||
      (st = view_packed(dD, KDA_F32, {a.C}, true, &dd, &s_dd)) != KDA_OK ||
      (dz && (st = view_rows(dz, a.dt, a.T, 0, a.C, true, &vdz)) != KDA_OK) ||
      (st = view_packed(ddt_bias, KDA_F32, {a.C}, true, &dbias, &s_dbias)) != KDA_OK ||
      (st = view_packed(dinitial_state, KDA_F32, {num_seqs, a.C, a.N}, true, &dinit, &s_dinit)) != KDA_OK)
    return st;
  if (any_overlap({vdu.span, vddt.span, s_da, vdb.span, vdc.span, s_dd, vdz.span, s_dbias, s_dinit},
                  {a.u.span, a.dt_.span, a.b.span, a.c.span, a.z.span, a.out.span, a.s_A, a.s_D, a.s_bias, s_init,
                   s_dfin}))
    return KDA_ERR_OVERLAP;
  int dev = 0;
  if ((st = prologue(&dev)) != KDA_OK) return st;
  if ((st = prepare_pool(dev)) != KDA_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  sm::BwdParams p;
  std::memset(&p, 0, sizeof(p));
  p.f = ssm_params(a, dt_softplus != 0, cu_seqlens, num_seqs, init);
  const int ch = sm::bwd_channels(static_cast<int>(a.N));
  p.f.blocks_per_group = static_cast<int>((a.C / a.G + ch - 1) / ch);
  const int64_t blocks = a.G * p.f.blocks_per_group;
  const size_t cn = static_cast<size_t>(a.C) * a.N;
  const int sms = g_num_sms[dev];
  p.f.run = split_run(a, num_seqs, blocks, {sm::bwd_resident(static_cast<int>(a.N)), 64, 40, 60, 1.35f, 2.16f}, dev);
  const int ranges = p.f.run ? static_cast<int>((a.T + p.f.run - 1) / p.f.run) : num_seqs;
  const size_t ck_bytes = round256((static_cast<size_t>(a.T) / sm::KT + num_seqs) * cn * 4);
  const size_t a_bytes = round256(ranges * cn * 4), d_bytes = round256(2 * static_cast<size_t>(ranges) * a.C * 4);
  const size_t carry_bytes = p.f.run ? a_bytes : 0, sum_bytes = p.f.run ? round256(static_cast<size_t>(ranges) * a.C * 4) : 0;
  const size_t b_bytes = round256(static_cast<size_t>(blocks) * a.T * a.N * 4);
  void* scratch = nullptr;
  cudaError_t e =
      pool_alloc(&scratch, ck_bytes + a_bytes + d_bytes + 2 * b_bytes + 2 * carry_bytes + sum_bytes, dev, cs);
  if (e != cudaSuccess) return cuda_fail(e);
  unsigned char* sb = static_cast<unsigned char*>(scratch);
  p.f.ck = reinterpret_cast<float*>(sb);
  p.part_a = reinterpret_cast<float*>(sb + ck_bytes);
  p.part_d = reinterpret_cast<float*>(sb + ck_bytes + a_bytes);
  p.part_b = reinterpret_cast<float*>(sb + ck_bytes + a_bytes + d_bytes);
  p.part_c = reinterpret_cast<float*>(sb + ck_bytes + a_bytes + d_bytes + b_bytes);
  if (p.f.run) {
    unsigned char* split = sb + ck_bytes + a_bytes + d_bytes + 2 * b_bytes;
    p.f.carry = reinterpret_cast<float*>(split);
    p.f.back = reinterpret_cast<float*>(split + carry_bytes);
    p.f.sum_d = reinterpret_cast<float*>(split + 2 * carry_bytes);
  }
  p.f.dout = a.out.data;
  p.f.dout_st = a.out.st;
  p.f.dfin = static_cast<const float*>(dfin);
  p.du = vdu.data;
  p.ddt = vddt.data;
  p.dz = vdz.data;
  p.du_st = vdu.st;
  p.ddt_st = vddt.st;
  p.dz_st = vdz.st;
  p.dinit = static_cast<float*>(dinit);
  sm::ReduceParams r;
  std::memset(&r, 0, sizeof(r));
  r.part_a = p.part_a;
  r.part_d = p.part_d;
  r.part_b = p.part_b;
  r.part_c = p.part_c;
  r.cu = cu_seqlens;
  r.dA = static_cast<float*>(da);
  r.dD = static_cast<float*>(dd);
  r.ddt_bias = static_cast<float*>(dbias);
  r.dB = vdb.data;
  r.dC = vdc.data;
  r.du = vdu.data;
  r.ddt = vddt.data;
  r.dz = vdz.data;
  r.T = a.T;
  r.dB_st = vdb.st;
  r.dB_sg = vdb.sg;
  r.dC_st = vdc.st;
  r.dC_sg = vdc.sg;
  r.du_st = vdu.st;
  r.ddt_st = vddt.st;
  r.dz_st = vdz.st;
  r.NS = num_seqs;
  r.parts = ranges;
  r.C = static_cast<int>(a.C);
  r.N = static_cast<int>(a.N);
  r.G = static_cast<int>(a.G);
  r.blocks_per_group = p.f.blocks_per_group;
  const int64_t most = std::max<int64_t>(a.T * a.G * a.N, static_cast<int64_t>(cn));
  const unsigned reduce_blocks =
      static_cast<unsigned>(std::min<int64_t>((most + 255) / 256, 8 * static_cast<int64_t>(g_num_sms[dev])));
  e = by_type(a.dt, dev, [&](auto m) {
    cudaError_t f = cudaSuccess;
    if (p.f.run && ranges > 1) {
      sm::Params first = p.f;
      first.ck = nullptr;
      f = m.scan(first, sm::STATES, ranges - 1, sms, cs);
      if (f == cudaSuccess) f = m.scan(first, sm::BACK, ranges - 1, sms, cs);
    }
    if (f == cudaSuccess) f = m.scan(p.f, sm::STATES, ranges, sms, cs);
    if (f == cudaSuccess) f = m.scan_bwd(p, ranges, cs);
    return f == cudaSuccess ? m.scan_reduce(r, reduce_blocks, cs) : f;
  });
  const cudaError_t ef = cudaFreeAsync(scratch, cs);
  if (e != cudaSuccess) return cuda_fail(e);
  return ef != cudaSuccess ? cuda_fail(ef) : KDA_OK;
}

}  // extern "C"
