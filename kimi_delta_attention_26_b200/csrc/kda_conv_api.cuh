// kda_conv_api.cuh -- argument checks shared by the convolution's and the
// scan's entry points, and the convolution's launches. Part of kda_api.cu's
// translation unit.
#pragma once

namespace {

// ------------------------------------------------------------ argument checks
// The memory of a tensor as rows: `width` bytes every `step` bytes.
struct Span {
  uintptr_t at;
  int64_t rows, step, width;
};

// Whether two tensors share a byte. Rows of equal steps may interleave (two
// column ranges of one buffer); other cases go by the whole extents.
bool overlap(const Span& a, const Span& b) {
  if (a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  const uintptr_t a1 = a.at + (a.rows - 1) * a.step + a.width, b1 = b.at + (b.rows - 1) * b.step + b.width;
  if (a1 <= b.at || b1 <= a.at) return false;
  if (a.rows > 1 && b.rows > 1 && a.step == b.step) {
    const int64_t step = a.step;
    int64_t d = static_cast<int64_t>(b.at - a.at) % step;
    if (d < 0) d += step;
    return !(d >= a.width && step - d >= b.width);
  }
  return true;
}

int io_bytes(kda_dtype_t dt) { return dt == KDA_F32 ? 4 : dt == KDA_BF16 || dt == KDA_F16 ? 2 : 0; }

// A tensor of token rows: [T, C] (G = 0) or [T, G, C]. Every type, any
// positive strides over tokens and groups, unit stride within a row; what is
// written may not overlap itself. Strides of dimensions of one element do not matter.
struct RowView {
  void* data = nullptr;
  int64_t st = 0, sg = 0;
  int eb = 1;               // bytes per element
  Span span{0, 0, 0, 0};
};

kda_status_t view_rows(const kda_tensor_t* t, kda_dtype_t dt, int64_t T, int64_t G, int64_t C, bool written, RowView* v) {
  if (!t) return KDA_ERR_NULL;
  if (t->dtype != dt) return KDA_ERR_DTYPE;
  const int last = G ? 2 : 1;
  if (t->ndim != last + 1 || t->shape[0] != T || t->shape[last] != C || (G && t->shape[1] != G)) return KDA_ERR_SHAPE;
  *v = RowView();
  if (T == 0) return KDA_OK;  // nothing is read or written
  const int eb = io_bytes(dt);
  if (C > 1 && t->stride[last] != 1) return KDA_ERR_STRIDE;
  v->sg = G > 1 ? t->stride[1] : 0;
  const int64_t limit = (int64_t(1) << 40) / eb;
  if (G > 1 && (v->sg <= 0 || v->sg >= limit)) return KDA_ERR_STRIDE;
  const int64_t extent = (G > 1 ? (G - 1) * v->sg : 0) + C;
  v->st = T > 1 ? t->stride[0] : extent;
  if (v->st <= 0 || v->st >= limit) return KDA_ERR_STRIDE;
  if (written && ((G > 1 && v->sg < C) || (T > 1 && v->st < extent))) return KDA_ERR_STRIDE;
  if (!t->data) return KDA_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(t->data) % eb != 0) return KDA_ERR_ALIGN;
  v->data = t->data;
  v->eb = eb;
  v->span = {reinterpret_cast<uintptr_t>(t->data), T, v->st * eb, extent * eb};
  return KDA_OK;
}

// A contiguous tensor; absent tensors pass where they are optional.
kda_status_t view_packed(const kda_tensor_t* t, kda_dtype_t dt, std::initializer_list<int64_t> shape, bool optional,
                         void** data, Span* span = nullptr) {
  *data = nullptr;
  if (span) *span = {0, 0, 0, 0};
  if (!t) return optional ? KDA_OK : KDA_ERR_NULL;
  if (t->dtype != dt) return KDA_ERR_DTYPE;
  if (t->ndim != static_cast<int32_t>(shape.size())) return KDA_ERR_SHAPE;
  int64_t n = 1;
  int i = 0;
  for (int64_t s : shape) {
    if (t->shape[i++] != s) return KDA_ERR_SHAPE;
    n *= s;
  }
  if (n == 0) return KDA_OK;
  int64_t want = 1;
  for (i = t->ndim - 1; i >= 0; --i) {
    if (t->shape[i] > 1 && t->stride[i] != want) return KDA_ERR_STRIDE;
    want *= t->shape[i];
  }
  if (!t->data) return KDA_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(t->data) % io_bytes(dt) != 0) return KDA_ERR_ALIGN;
  *data = t->data;
  if (span) *span = {reinterpret_cast<uintptr_t>(t->data), 1, n * io_bytes(dt), n * io_bytes(dt)};
  return KDA_OK;
}

bool any_overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (overlap(*o, i)) return true;
    for (const Span* q = o + 1; q != outs.end(); ++q)
      if (overlap(*o, *q)) return true;
  }
  return false;
}

constexpr int64_t kMaxRows = int64_t(INT32_MAX) - 256;  // boundaries are 32-bit

kda_status_t check_packing_args(const int32_t* cu, int32_t num_seqs, int64_t T) {
  if (T < 0 || T > kMaxRows || num_seqs < 1 || num_seqs > 65535 || (!cu && num_seqs != 1)) return KDA_ERR_SHAPE;
  if (reinterpret_cast<uintptr_t>(cu) & 3u) return KDA_ERR_ALIGN;
  return KDA_OK;
}

// The rows of `v` start at multiples of `bytes`.
bool aligned(const RowView& v, int64_t bytes) {
  return v.span.at % bytes == 0 && v.span.step % bytes == 0 && v.sg * v.eb % bytes == 0;
}
bool aligned(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Bit dt: a kernel of that element type's translation unit may have run on the
// device, so that its status words count. The others' are 0, and reading them
// would load that unit's code onto the device (13 ms each).
std::atomic<uint32_t> g_mixer_used[kMaxDevices];

// f(the launches of the type)
template <typename F>
cudaError_t by_type(kda_dtype_t dt, int dev, F f) {
  const uint32_t bit = 1u << dt;
  if (!(g_mixer_used[dev].load(std::memory_order_relaxed) & bit)) g_mixer_used[dev].fetch_or(bit);
  if (dt == KDA_BF16) return f(kda::Mixer<__nv_bfloat16>());
  if (dt == KDA_F16) return f(kda::Mixer<__half>());
  return f(kda::Mixer<float>());
}

// ------------------------------------------------------------- convolution
constexpr int64_t kConvMaxChannels = 1 << 20;

struct ConvArgs {
  int64_t T, C;
  int W;
  kda_dtype_t dt;
  RowView x, out;           // out: dout for the backward pass
  void *weight, *bias;
  Span weight_span, bias_span;
};

kda_status_t check_conv(const kda_tensor_t* x, const kda_tensor_t* weight, const kda_tensor_t* bias, int32_t activation,
                        const kda_tensor_t* out, bool written, ConvArgs* a) {
  if (!x || !weight || !out) return KDA_ERR_NULL;
  if (!io_bytes(x->dtype)) return KDA_ERR_DTYPE;
  if (x->ndim != 2 || weight->ndim != 2) return KDA_ERR_SHAPE;
  a->dt = x->dtype;
  a->T = x->shape[0];
  a->C = x->shape[1];
  const int64_t W = weight->shape[1];
  if (a->T < 0 || a->T > kMaxRows || a->C < 1 || a->C > kConvMaxChannels || W < 2 || W > 4) return KDA_ERR_SHAPE;
  a->W = static_cast<int>(W);
  if (activation != KDA_ACT_NONE && activation != KDA_ACT_SILU) return KDA_ERR_VALUE;
  kda_status_t st;
  if ((st = view_rows(x, a->dt, a->T, 0, a->C, false, &a->x)) != KDA_OK ||
      (st = view_packed(weight, KDA_F32, {a->C, W}, false, &a->weight, &a->weight_span)) != KDA_OK ||
      (st = view_packed(bias, KDA_F32, {a->C}, true, &a->bias, &a->bias_span)) != KDA_OK ||
      (st = view_rows(out, a->dt, a->T, 0, a->C, written, &a->out)) != KDA_OK)
    return st;
  return KDA_OK;
}

// Tokens per warp: enough warps to fill the device, in steps of `unit` tokens
// and at most `most`.
int64_t conv_run(int64_t T, int64_t channel_blocks, int dev, int unit, int most) {
  const int64_t warps = static_cast<int64_t>(g_num_sms[dev]) * 32;
  const int64_t per = T * channel_blocks / warps;
  return std::max<int64_t>(unit, std::min<int64_t>(most, per / unit * unit));
}

}  // namespace

extern "C" {

kda_status_t kda_conv_fwd(const kda_tensor_t* x, const kda_tensor_t* weight, const kda_tensor_t* bias,
                          int32_t activation, const int32_t* cu_seqlens, int32_t num_seqs,
                          const kda_tensor_t* initial_state, const kda_tensor_t* out, const kda_tensor_t* final_state,
                          void* stream) {
  namespace cv = kda::conv;
  g_last_cuda_error[0] = '\0';
  ConvArgs a;
  kda_status_t st = check_conv(x, weight, bias, activation, out, true, &a);
  if (st != KDA_OK) return st;
  if ((st = check_packing_args(cu_seqlens, num_seqs, a.T)) != KDA_OK) return st;
  void *init, *fin;
  Span s_init, s_fin;
  if ((st = view_packed(initial_state, a.dt, {num_seqs, a.W - 1, a.C}, true, &init, &s_init)) != KDA_OK ||
      (st = view_packed(final_state, a.dt, {num_seqs, a.W - 1, a.C}, true, &fin, &s_fin)) != KDA_OK)
    return st;
  if (any_overlap({a.out.span, s_fin}, {a.x.span, s_init, a.weight_span, a.bias_span})) return KDA_ERR_OVERLAP;
  int dev = 0;
  if ((st = prologue(&dev)) != KDA_OK) return st;
  constexpr int RB = cv::RUN_BYTES;
  const int V = RB / io_bytes(a.dt);
  const bool vec = a.C % V == 0 && aligned(a.x, RB) && aligned(a.out, RB) && aligned(init, RB) && aligned(fin, RB);
  const int64_t cb = (a.C + 32 * (vec ? V : 1) - 1) / (32 * (vec ? V : 1));
  cv::Params p;
  p.x = a.x.data;
  p.weight = static_cast<const float*>(a.weight);
  p.bias = static_cast<const float*>(a.bias);
  p.cu = cu_seqlens;
  p.init = init;
  p.out = a.out.data;
  p.fin = fin;
  p.T = a.T;
  p.C = a.C;
  p.x_st = a.x.st;
  p.o_st = a.out.st;
  p.run = conv_run(a.T, cb, dev, 8, 128);
  p.run_blocks = (a.T + p.run * cv::NWARPS - 1) / (p.run * cv::NWARPS);
  p.N = num_seqs;
  p.silu = activation == KDA_ACT_SILU;
  const dim3 grid(static_cast<unsigned>(p.run_blocks + (num_seqs + cv::NWARPS - 1) / cv::NWARPS), static_cast<unsigned>(cb));
  const cudaError_t e = by_type(a.dt, dev, [&](auto m) { return m.conv_fwd(p, a.W, vec, grid, static_cast<cudaStream_t>(stream)); });
  return e != cudaSuccess ? cuda_fail(e) : KDA_OK;
}

kda_status_t kda_conv_decode(const kda_tensor_t* x, const kda_tensor_t* weight, const kda_tensor_t* bias,
                             int32_t activation, const kda_tensor_t* state, const int32_t* state_indices,
                             const kda_tensor_t* out, void* stream) {
  namespace cv = kda::conv;
  g_last_cuda_error[0] = '\0';
  ConvArgs a;
  kda_status_t st = check_conv(x, weight, bias, activation, out, true, &a);
  if (st != KDA_OK) return st;
  if (!state) return KDA_ERR_NULL;
  if (state->ndim != 3) return KDA_ERR_SHAPE;
  const int64_t B = a.T, pool = state->shape[0];
  if (pool < 1 || (!state_indices && pool < B)) return KDA_ERR_SHAPE;
  if (pool > (int64_t(1) << 40) / a.C) return KDA_ERR_SHAPE;
  void* sp;
  Span s_state;
  if ((st = view_packed(state, a.dt, {pool, a.W - 1, a.C}, false, &sp, &s_state)) != KDA_OK) return st;
  if (reinterpret_cast<uintptr_t>(state_indices) & 3u) return KDA_ERR_ALIGN;
  // a thread reads its token before it writes the output: they may be the same tensor
  const bool in_place = a.out.data == a.x.data && a.out.st == a.x.st;
  if (any_overlap({a.out.span, s_state}, {a.weight_span, a.bias_span}) || overlap(s_state, a.x.span) ||
      (!in_place && overlap(a.out.span, a.x.span)))
    return KDA_ERR_OVERLAP;
  int dev = 0;
  if ((st = prologue(&dev)) != KDA_OK) return st;
  if (B == 0) return KDA_OK;
  constexpr int RB = cv::RUN_BYTES;
  const int V = RB / io_bytes(a.dt);
  const bool vec = a.C % V == 0 && aligned(a.x, RB) && aligned(a.out, RB) && aligned(sp, RB);
  cv::DecodeParams p;
  p.x = a.x.data;
  p.weight = static_cast<const float*>(a.weight);
  p.bias = static_cast<const float*>(a.bias);
  p.state = sp;
  p.idx = state_indices;
  p.out = a.out.data;
  p.B = B;
  p.C = a.C;
  p.x_st = a.x.st;
  p.o_st = a.out.st;
  p.pool = pool;
  p.silu = activation == KDA_ACT_SILU;
  // enough blocks to fill the device; each takes every grid.y-th request
  const int per = cv::NTHREADS * (vec ? V : 1);
  const int64_t cb = (a.C + per - 1) / per, rows = std::max<int64_t>(1, int64_t(8) * g_num_sms[dev] / cb);
  const dim3 grid(static_cast<unsigned>(cb), static_cast<unsigned>(std::min({B, rows, int64_t(65535)})));
  const cudaError_t e = by_type(a.dt, dev, [&](auto m) { return m.conv_decode(p, a.W, vec, grid, static_cast<cudaStream_t>(stream)); });
  return e != cudaSuccess ? cuda_fail(e) : KDA_OK;
}

kda_status_t kda_conv_bwd(const kda_tensor_t* x, const kda_tensor_t* weight, const kda_tensor_t* bias,
                          int32_t activation, const int32_t* cu_seqlens, int32_t num_seqs,
                          const kda_tensor_t* initial_state, const kda_tensor_t* dout, const kda_tensor_t* dfinal_state,
                          const kda_tensor_t* dx, const kda_tensor_t* dweight, const kda_tensor_t* dbias,
                          const kda_tensor_t* dinitial_state, void* stream) {
  namespace cv = kda::conv;
  g_last_cuda_error[0] = '\0';
  ConvArgs a;
  kda_status_t st = check_conv(x, weight, bias, activation, dout, false, &a);
  if (st != KDA_OK) return st;
  if ((st = check_packing_args(cu_seqlens, num_seqs, a.T)) != KDA_OK) return st;
  RowView g;
  void *init, *dfin, *dinit, *dw, *db;
  Span s_init, s_dfin, s_dinit, s_dw, s_db;
  if ((st = view_packed(initial_state, a.dt, {num_seqs, a.W - 1, a.C}, true, &init, &s_init)) != KDA_OK ||
      (st = view_packed(dfinal_state, a.dt, {num_seqs, a.W - 1, a.C}, true, &dfin, &s_dfin)) != KDA_OK ||
      (st = view_rows(dx, a.dt, a.T, 0, a.C, true, &g)) != KDA_OK ||
      (st = view_packed(dweight, KDA_F32, {a.C, a.W}, false, &dw, &s_dw)) != KDA_OK ||
      (st = view_packed(dbias, KDA_F32, {a.C}, true, &db, &s_db)) != KDA_OK ||
      (st = view_packed(dinitial_state, a.dt, {num_seqs, a.W - 1, a.C}, true, &dinit, &s_dinit)) != KDA_OK)
    return st;
  if (any_overlap({g.span, s_dw, s_db, s_dinit},
                  {a.x.span, a.out.span, s_init, s_dfin, a.weight_span, a.bias_span}))
    return KDA_ERR_OVERLAP;
  int dev = 0;
  if ((st = prologue(&dev)) != KDA_OK) return st;
  if ((st = prepare_pool(dev)) != KDA_OK) return st;
  constexpr int RB = cv::RUN_BYTES;
  const int V = RB / io_bytes(a.dt);
  const bool vec = a.C % V == 0 && aligned(a.x, RB) && aligned(a.out, RB) && aligned(g, RB) && aligned(init, RB) &&
                   aligned(dfin, RB) && aligned(dinit, RB);
  const int64_t cb = (a.C + 32 * (vec ? V : 1) - 1) / (32 * (vec ? V : 1));
  cv::BwdParams p;
  p.x = a.x.data;
  p.dout = a.out.data;
  p.weight = static_cast<const float*>(a.weight);
  p.bias = static_cast<const float*>(a.bias);
  p.cu = cu_seqlens;
  p.init = init;
  p.dfin = dfin;
  p.dx = g.data;
  p.dinit = dinit;
  p.T = a.T;
  p.C = a.C;
  p.x_st = a.x.st;
  p.d_st = a.out.st;
  p.g_st = g.st;
  p.run = conv_run(a.T, cb, dev, 16, 256);
  p.run_blocks = (a.T + p.run * cv::NWARPS - 1) / (p.run * cv::NWARPS);
  p.N = num_seqs;
  p.silu = activation == KDA_ACT_SILU;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  void* part = nullptr;
  cudaError_t e = pool_alloc(&part, (p.run_blocks + 1) * (a.W + 1) * a.C * sizeof(float), dev, cs);
  if (e != cudaSuccess) return cuda_fail(e);
  p.part = static_cast<float*>(part);
  const dim3 grid(static_cast<unsigned>(p.run_blocks + (num_seqs + cv::NWARPS - 1) / cv::NWARPS), static_cast<unsigned>(cb));
  e = by_type(a.dt, dev, [&](auto m) { return m.conv_bwd(p, a.W, vec, grid, cs); });
  if (e == cudaSuccess) {
    cv::conv_reduce_kernel<<<dim3(static_cast<unsigned>((a.C + cv::NTHREADS - 1) / cv::NTHREADS), a.W + 1), cv::NTHREADS, 0, cs>>>(
      p.part, p.run_blocks, a.W, a.C, static_cast<float*>(dw), static_cast<float*>(db));
    e = cudaGetLastError();
  }
  const cudaError_t ef = cudaFreeAsync(part, cs);
  if (e != cudaSuccess) return cuda_fail(e);
  return ef != cudaSuccess ? cuda_fail(ef) : KDA_OK;
}

}  // extern "C"
