// gdp_recurrence.cu -- the gated linear recurrence (gdp_layer.h): C entries, argument checks, and the
// one-token step.  The scans over packed sequences are in gdp_rec_fwd_body.cuh and gdp_rec_bwd_body.cuh.
#include <atomic>

#include "gdp_rec_scan.cuh"

namespace gdp {
namespace layer {
namespace {

constexpr int kThreads = 128;

struct RecProblem {
  const void *x, *g;
  int64_t x_st, g_st;
  void *h;
  const void *cu;
  int cu64;
  int64_t T, N, C;
  const float *init;
  float *fin;
  float *cache;
  const int32_t *slots;
  int64_t num_slots;
  uint32_t *status;
  int x_type, g_type, gate;
};

// The state row of sequence i: where it is read (NULL: zero) and written (NULL: nowhere).
__device__ __forceinline__ void state_rows(const RecProblem &p, int64_t i, bool report, const float **src, float **dst) {
  *src = p.init ? p.init + i * p.C : nullptr;
  *dst = p.fin ? p.fin + i * p.C : nullptr;
  if (p.cache) {
    int64_t slot = p.slots[i];
    if (slot < -1 || slot >= p.num_slots) {
      if (report) set_status(p.status, GDP_DEV_ERR_SLOT);
      slot = -1;
    }
    *src = *dst = slot >= 0 ? p.cache + slot * p.C : nullptr;
  }
}

// Four values of a row: 16 bytes of fp32, 8 of a 16-bit type.
template <typename T>
struct alignas(4 * sizeof(T)) Quad {
  T v[4];
};

// The one-token step: every value is touched once, so it is bound by memory, and at serving sizes by its
// own latency (64 x 2048 bf16: 1.7 MB in 2.2 us on the device, 0.25 us at the memory's rate).  VEC channels
// per thread (4 where rows are aligned, else 1).
template <typename TX, typename TG, int VEC>
__global__ void __launch_bounds__(kThreads) gdp_rec_step_kernel(const RecProblem p) {
  const int64_t i = blockIdx.x, c = ((int64_t)blockIdx.y * kThreads + threadIdx.x) * VEC;
  if (c >= p.C) return;
  const float *src;
  float *dst;
  const TX *x_at = static_cast<const TX *>(p.x) + i * p.x_st + c;
  const TG *g_at = static_cast<const TG *>(p.g) + i * p.g_st + c;
  TX *h_at = static_cast<TX *>(p.h) + i * p.C + c;
  auto one = [&](float x, float g, float s) {
    float a, f;
    if (p.gate == GDP_GATE_LOG) gate_eval<GDP_GATE_LOG>(g, &a, &f);
    else if (p.gate == GDP_GATE_ALPHA) gate_eval<GDP_GATE_ALPHA>(g, &a, &f);
    else gate_eval<GDP_GATE_SIGMOID>(g, &a, &f);
    return fmaf(a, s, f * x);
  };
  if constexpr (VEC == 4) {
    const Quad<TX> x = *reinterpret_cast<const Quad<TX> *>(x_at);
    const Quad<TG> g = *reinterpret_cast<const Quad<TG> *>(g_at);
    state_rows(p, i, c == 0, &src, &dst);
    const float4 s = src ? *reinterpret_cast<const float4 *>(src + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 h = make_float4(one(to_f32(x.v[0]), to_f32(g.v[0]), s.x), one(to_f32(x.v[1]), to_f32(g.v[1]), s.y),
                                 one(to_f32(x.v[2]), to_f32(g.v[2]), s.z), one(to_f32(x.v[3]), to_f32(g.v[3]), s.w));
    *reinterpret_cast<Quad<TX> *>(h_at) = Quad<TX>{{from_f32<TX>(h.x), from_f32<TX>(h.y), from_f32<TX>(h.z), from_f32<TX>(h.w)}};
    if (dst) *reinterpret_cast<float4 *>(dst + c) = h;
  } else {
    const float x = to_f32(*x_at), g = to_f32(*g_at);
    state_rows(p, i, c == 0, &src, &dst);
    const float h = one(x, g, src ? src[c] : 0.f);
    *h_at = from_f32<TX>(h);
    if (dst) dst[c] = h;
  }
}

template <typename TX, typename TG>
void launch_step(const RecProblem &p, cudaStream_t stream) {
  const bool vec = p.C % 4 == 0 && p.x_st % 4 == 0 && p.g_st % 4 == 0 && aligned(p.x, 4 * sizeof(TX)) && aligned(p.g, 4 * sizeof(TG)) &&
                   aligned(p.h, 4 * sizeof(TX)) && aligned(p.init, 16) && aligned(p.fin, 16) && aligned(p.cache, 16);
  const int64_t width = vec ? 4 : 1;
  const dim3 grid((unsigned)p.N, (unsigned)((p.C + kThreads * width - 1) / (kThreads * width)));
  if (vec) gdp_rec_step_kernel<TX, TG, 4><<<grid, kThreads, 0, stream>>>(p);
  else gdp_rec_step_kernel<TX, TG, 1><<<grid, kThreads, 0, stream>>>(p);
}

gdp_status check_shape(int64_t T, int64_t N, int64_t C, int x_type, int g_type, int gate) {
  if (T < 0 || N < 0 || C < 1) return fail(GDP_ERR_INVALID_ARG, "T >= 0, N >= 0 and C >= 1 are required");
  if (T > INT32_MAX || N > INT32_MAX || C > (1 << 20)) return fail(GDP_ERR_UNSUPPORTED, "T and N below 2^31, C up to 2^20");
  if (!dtype_ok(x_type)) return fail(GDP_ERR_UNSUPPORTED, "x_dtype must be GDP_DTYPE_BF16, GDP_DTYPE_F16 or GDP_DTYPE_F32");
  if (g_type != x_type && g_type != GDP_DTYPE_F32) return fail(GDP_ERR_UNSUPPORTED, "g_dtype must be x_dtype or GDP_DTYPE_F32");
  if (gate != GDP_GATE_LOG && gate != GDP_GATE_ALPHA && gate != GDP_GATE_SIGMOID)
    return fail(GDP_ERR_INVALID_ARG, "gate must be GDP_GATE_LOG, GDP_GATE_ALPHA or GDP_GATE_SIGMOID");
  return GDP_OK;
}

// A [T, C] tensor: given where it has elements, aligned to its elements, rows at least C apart.
gdp_status check_rows(const void *p, int64_t stride, int64_t T, int64_t C, int type, const char *name) {
  const size_t es = dtype_size(type);
  if (T > 0 && !p) {
    set_last_error("%s is required", name);
    return GDP_ERR_INVALID_ARG;
  }
  if (!aligned(p, es) || (T > 1 && stride < C)) {
    set_last_error("%s must be aligned to its elements, its rows at least C elements apart", name);
    return GDP_ERR_INVALID_ARG;
  }
  return GDP_OK;
}

// The stride of a single row means nothing and may be anything in a view (a tensor map refuses 0): one that fits.
int64_t row_stride(int64_t stride, int64_t T, int64_t C) { return T > 1 ? stride : (C + 15) / 16 * 16; }

gdp_status resolve(const gdp_recurrence_args *a, bool step, RecProblem *p) {
  set_last_error("");
  if (!a) return fail(GDP_ERR_INVALID_ARG, "args is NULL");
  gdp_status st = check_shape(a->T, a->N, a->C, a->x_dtype, a->g_dtype, a->gate);
  if (st != GDP_OK) return st;
  if (step && a->T != a->N) return fail(GDP_ERR_INVALID_ARG, "decode takes one token per sequence: T == N");
  if ((st = check_rows(a->x, a->x_stride_t, a->T, a->C, a->x_dtype, "x")) != GDP_OK) return st;
  if ((st = check_rows(a->g, a->g_stride_t, a->T, a->C, a->g_dtype, "g")) != GDP_OK) return st;
  if ((st = check_rows(a->output, a->C, a->T, a->C, a->x_dtype, "output")) != GDP_OK) return st;
  if (!step && !a->cu_seqlens) return fail(GDP_ERR_INVALID_ARG, "cu_seqlens is required");
  if (!aligned(a->initial_state, 4) || !aligned(a->output_state, 4) || !aligned(a->state, 4) || !aligned(a->state_indices, 4))
    return fail(GDP_ERR_INVALID_ARG, "state buffers must be 4-byte aligned");
  if (a->state && (a->initial_state || a->output_state))
    return fail(GDP_ERR_INVALID_ARG, "the state cache excludes initial_state and output_state");
  if (a->state && (!a->state_indices || a->num_slots < 1))
    return fail(GDP_ERR_INVALID_ARG, "the state cache needs state_indices and num_slots >= 1");
  if (partly_overlap(a->initial_state, a->output_state, sizeof(float) * (size_t)a->N * (size_t)a->C))
    return fail(GDP_ERR_ALIAS, "output_state partly overlaps initial_state");
  *p = RecProblem{a->x, a->g, row_stride(a->x_stride_t, a->T, a->C), row_stride(a->g_stride_t, a->T, a->C), a->output, a->cu_seqlens, a->cu_seqlens_int64 != 0, a->T, a->N, a->C,
                  a->initial_state, a->output_state, a->state, a->state_indices, a->num_slots, a->device_status,
                  a->x_dtype, a->g_dtype, a->gate};
  return GDP_OK;
}

// A [T, C] output none of whose rows belongs to a sequence.
gdp_status zero_rows(void *p, int64_t T, int64_t C, int type, cudaStream_t stream) {
  if (T == 0) return GDP_OK;
  const cudaError_t e = cudaMemsetAsync(p, 0, (size_t)T * (size_t)C * dtype_size(type), stream);
  if (e == cudaSuccess) return GDP_OK;
  set_last_error("recurrence padding rows: %s", cudaGetErrorString(e));
  return GDP_ERR_CUDA;
}

// Set by gdp_arm_recurrence_wait_test for the calling thread's next scan.
thread_local uint64_t armed_limit_ns = 0;

void set_limits(ScanShape &s) {
  s.limit_ns = armed_limit_ns ? armed_limit_ns : sm100::kWaitLimitNs;
  s.withhold = armed_limit_ns != 0;
  armed_limit_ns = 0;
}

cudaError_t run(RecFwd &p, int gate, cudaStream_t stream, bool bf16, bool wide) {
  if (bf16) return wide ? launch_rec_fwd<__nv_bfloat16, float>(p, gate, stream) : launch_rec_fwd<__nv_bfloat16, __nv_bfloat16>(p, gate, stream);
  return wide ? launch_rec_fwd<__half, float>(p, gate, stream) : launch_rec_fwd<__half, __half>(p, gate, stream);
}
cudaError_t run(RecBwd &p, int gate, cudaStream_t stream, bool bf16, bool wide) {
  if (bf16) return wide ? launch_rec_bwd<__nv_bfloat16, float>(p, gate, stream) : launch_rec_bwd<__nv_bfloat16, __nv_bfloat16>(p, gate, stream);
  return wide ? launch_rec_bwd<__half, float>(p, gate, stream) : launch_rec_bwd<__half, __half>(p, gate, stream);
}
cudaError_t run_f32(RecFwd &p, int gate, cudaStream_t stream) { return launch_rec_fwd<float, float>(p, gate, stream); }
cudaError_t run_f32(RecBwd &p, int gate, cudaStream_t stream) { return launch_rec_bwd<float, float>(p, gate, stream); }

template <typename P>
gdp_status dispatch(int x_type, int g_type, P &p, int gate, cudaStream_t stream) {
  const cudaError_t e = x_type == GDP_DTYPE_F32 ? run_f32(p, gate, stream)
                                                : run(p, gate, stream, x_type == GDP_DTYPE_BF16, g_type == GDP_DTYPE_F32);
  if (e == cudaSuccess) return GDP_OK;
  set_last_error("recurrence kernel: %s", cudaGetErrorString(e));
  return GDP_ERR_CUDA;
}

}  // namespace

int sm_count() {
  static std::atomic<int> counts[64];  // (host threads may ask at once)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  int n = counts[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 152;
    counts[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

}  // namespace layer
}  // namespace gdp

GDP_EXPORT gdp_status gdp_linear_recurrence(const gdp_recurrence_args *args, void *stream) {
  using namespace gdp::layer;
  RecProblem p;
  const gdp_status st = resolve(args, false, &p);
  if (st != GDP_OK) return st;
  if (p.N == 0) return args->zero_padding ? zero_rows(p.h, p.T, p.C, p.x_type, (cudaStream_t)stream) : GDP_OK;
  RecFwd f{};
  f.s.cu = p.cu; f.s.cu64 = p.cu64; f.s.T = p.T; f.s.N = p.N; f.s.C = p.C;
  f.s.slots = p.cache ? p.slots : nullptr; f.s.num_slots = p.num_slots; f.s.status = p.status;
  f.s.zero_pad = args->zero_padding != 0;
  set_limits(f.s);
  f.x = {p.x, p.x_st}; f.g = {p.g, p.g_st}; f.h = p.h;
  f.from = p.cache ? p.cache : p.init;
  f.to = p.cache ? p.cache : p.fin;
  f.pair_out = p.C % 2 == 0 && aligned(p.h, 2 * dtype_size(p.x_type));
  return dispatch(p.x_type, p.g_type, f, p.gate, (cudaStream_t)stream);
}

GDP_EXPORT gdp_status gdp_linear_recurrence_decode(const gdp_recurrence_args *args, void *stream) {
  using namespace gdp::layer;
  RecProblem p;
  const gdp_status st = resolve(args, true, &p);
  if (st != GDP_OK || p.N == 0) return st;
  const bool wide = p.g_type == GDP_DTYPE_F32;
  cudaStream_t s = (cudaStream_t)stream;
  if (p.x_type == GDP_DTYPE_F32) launch_step<float, float>(p, s);
  else if (p.x_type == GDP_DTYPE_BF16 && wide) launch_step<__nv_bfloat16, float>(p, s);
  else if (p.x_type == GDP_DTYPE_BF16) launch_step<__nv_bfloat16, __nv_bfloat16>(p, s);
  else if (wide) launch_step<__half, float>(p, s);
  else launch_step<__half, __half>(p, s);
  return launch_status("recurrence step kernel");
}

GDP_EXPORT gdp_status gdp_linear_recurrence_backward(const gdp_recurrence_backward_args *a, void *stream) {
  using namespace gdp::layer;
  gdp::set_last_error("");
  if (!a) return fail(GDP_ERR_INVALID_ARG, "args is NULL");
  gdp_status st = check_shape(a->T, a->N, a->C, a->x_dtype, a->g_dtype, a->gate);
  if (st != GDP_OK) return st;
  if ((st = check_rows(a->g, a->g_stride_t, a->T, a->C, a->g_dtype, "g")) != GDP_OK) return st;
  if ((st = check_rows(a->d_output, a->d_output_stride_t, a->T, a->C, a->x_dtype, "d_output")) != GDP_OK) return st;
  if (a->gate == GDP_GATE_SIGMOID && (st = check_rows(a->x, a->x_stride_t, a->T, a->C, a->x_dtype, "x")) != GDP_OK) return st;
  if ((st = check_rows(a->dx, a->C, a->T, a->C, a->x_dtype, "dx")) != GDP_OK) return st;
  if ((st = check_rows(a->dg, a->C, a->T, a->C, a->g_dtype, "dg")) != GDP_OK) return st;
  if (a->T > 0 && (a->h != nullptr) == (a->h_codes != nullptr))
    return fail(GDP_ERR_INVALID_ARG, "exactly one of h and h_codes is required");
  if (a->h && (st = check_rows(a->h, a->h_stride_t, a->T, a->C, a->x_dtype, "h")) != GDP_OK) return st;
  if (a->h_codes && (!a->h_scales || !aligned(a->h_scales, 4) || a->h_group < 1 || a->C % a->h_group != 0))
    return fail(GDP_ERR_INVALID_ARG, "h_codes needs h_scales and an h_group that divides C");
  if (!a->cu_seqlens) return fail(GDP_ERR_INVALID_ARG, "cu_seqlens is required");
  if (!aligned(a->initial_state, 4) || !aligned(a->d_final_state, 4) || !aligned(a->d_initial_state, 4))
    return fail(GDP_ERR_INVALID_ARG, "state buffers must be 4-byte aligned");
  const size_t bytes = sizeof(float) * (size_t)a->N * (size_t)a->C;
  if (overlap(a->d_final_state, a->d_initial_state, bytes) || overlap(a->initial_state, a->d_initial_state, bytes))
    return fail(GDP_ERR_ALIAS, "d_initial_state overlaps initial_state or d_final_state");
  if (a->N == 0) {  // every row is padding
    st = zero_rows(a->dx, a->T, a->C, a->x_dtype, (cudaStream_t)stream);
    return st != GDP_OK ? st : zero_rows(a->dg, a->T, a->C, a->g_dtype, (cudaStream_t)stream);
  }
  RecBwd p{};
  p.s.cu = a->cu_seqlens; p.s.cu64 = a->cu_seqlens_int64 != 0; p.s.T = a->T; p.s.N = a->N; p.s.C = a->C;
  p.s.status = a->device_status;
  set_limits(p.s);
  auto rows_of = [&](const void *at, int64_t stride) { return RowSource{at, row_stride(stride, a->T, a->C)}; };
  p.g = rows_of(a->g, a->g_stride_t); p.x = rows_of(a->x, a->x_stride_t);
  p.h = rows_of(a->h, a->h_stride_t); p.dout = rows_of(a->d_output, a->d_output_stride_t);
  p.codes = {a->h_codes, a->C};
  p.scales = a->h_scales;
  p.group = a->h_codes ? a->h_group : 1;
  p.blocks = (p.group + kBlock - 1) / kBlock;
  p.init = a->initial_state; p.dfin = a->d_final_state;
  p.dx = a->dx; p.dg = a->dg; p.dinit = a->d_initial_state;
  p.pair_dx = a->C % 2 == 0 && aligned(a->dx, 2 * dtype_size(a->x_dtype));
  p.pair_dg = a->C % 2 == 0 && aligned(a->dg, 2 * dtype_size(a->g_dtype));
  return dispatch(a->x_dtype, a->g_dtype, p, a->gate, (cudaStream_t)stream);
}

GDP_EXPORT gdp_status gdp_arm_recurrence_wait_test(uint64_t limit_ns) {
  using namespace gdp::layer;
  gdp::set_last_error("");
  if (limit_ns < 100000ull || limit_ns > 1000000000ull) return fail(GDP_ERR_INVALID_ARG, "limit_ns must be between 1e5 and 1e9");
  armed_limit_ns = limit_ns;
  return GDP_OK;
}

GDP_EXPORT size_t gdp_layer_args_size(int which) {
  switch (which) {
    case 0: return sizeof(gdp_recurrence_args);
    case 1: return sizeof(gdp_recurrence_backward_args);
    case 2: return sizeof(gdp_group_norm_args);
    case 3: return sizeof(gdp_group_norm_backward_args);
    default: return 0;
  }
}
