// gdp_ssm.cu -- the selective state space scan's C entries and argument checks (gdp_block.h).
#include "gdp_ssm.cuh"

namespace gdp {
namespace layer {
namespace {

// The parts of the arguments that the calls share.
template <typename Args>
gdp_status common(const Args *a, SsmProblem *p) {
  gdp_status st = shape_ok(a->T, a->N, a->C);
  if (st != GDP_OK) return st;
  if (!dtype_ok(a->x_dtype)) return fail(GDP_ERR_UNSUPPORTED, "x_dtype must be GDP_DTYPE_BF16, GDP_DTYPE_F16 or GDP_DTYPE_F32");
  if (a->dt_dtype != a->x_dtype && a->dt_dtype != GDP_DTYPE_F32) return fail(GDP_ERR_UNSUPPORTED, "dt_dtype must be x_dtype or GDP_DTYPE_F32");
  if (a->S < 1 || a->G < 1 || a->C % a->G != 0) return fail(GDP_ERR_INVALID_ARG, "S >= 1 and a G that divides C are required");
  if (a->S > 64) return fail(GDP_ERR_UNSUPPORTED, "S up to 64");
  const int64_t per = a->C / a->G, tiles = ssm_tiles(per, a->S);
  if (a->G * tiles > 65535 || (a->N + 1) * a->G * tiles > INT32_MAX) return fail(GDP_ERR_UNSUPPORTED, "too many groups, or sequences by channels");
  if ((st = rows_ok(a->x, a->x_stride_t, a->T, a->C, a->x_dtype, "x")) != GDP_OK) return st;
  if ((st = rows_ok(a->dt, a->dt_stride_t, a->T, a->C, a->dt_dtype, "dt")) != GDP_OK) return st;
  if (a->z && (st = rows_ok(a->z, a->z_stride_t, a->T, a->C, a->x_dtype, "z")) != GDP_OK) return st;
  // a token's groups may overlap no other group's
  if ((st = rows_ok(a->B, a->B_stride_t, a->T, a->S, a->x_dtype, "B")) != GDP_OK) return st;
  if ((st = rows_ok(a->C_in, a->C_stride_t, a->T, a->S, a->x_dtype, "C")) != GDP_OK) return st;
  if (a->G > 1 && (a->B_stride_g < a->S || a->C_stride_g < a->S)) return fail(GDP_ERR_INVALID_ARG, "groups of B and C must be at least S apart");
  if (!a->A) return fail(GDP_ERR_INVALID_ARG, "A is required");
  if (!aligned(a->A, 4) || !aligned(a->D, 4) || !aligned(a->dt_bias, 4)) return fail(GDP_ERR_INVALID_ARG, "fp32 buffers must be 4-byte aligned");
  *p = SsmProblem{};
  p->x = a->x; p->dt = a->dt; p->z = a->z; p->B = a->B; p->Cm = a->C_in;
  p->x_st = stride_of(a->x_stride_t, a->T, a->C); p->dt_st = stride_of(a->dt_stride_t, a->T, a->C);
  p->z_st = stride_of(a->z_stride_t, a->T, a->C);
  p->B_st = stride_of(a->B_stride_t, a->T, a->S); p->C_st = stride_of(a->C_stride_t, a->T, a->S);
  p->B_sg = a->G > 1 ? a->B_stride_g : 0; p->C_sg = a->G > 1 ? a->C_stride_g : 0;
  p->A = a->A; p->D = a->D; p->bias = a->dt_bias;
  p->p = Packed{a->cu_seqlens, a->cu_seqlens_int64 != 0, a->T, a->N, a->device_status};
  p->C = a->C; p->S = a->S; p->G = a->G;
  p->per = per; p->tiles = (int)tiles;
  p->dt_f32 = a->dt_dtype == GDP_DTYPE_F32;
  p->softplus = a->dt_softplus != 0;
  p->sms = sm_count();
  const int es = dtype_size(a->x_dtype), ds = dtype_size(a->dt_dtype);
  // (a CTA's channels begin at a multiple of eight within their group)
  p->fast_rows = (a->G == 1 || per * es % 16 == 0) && a->C * es % 16 == 0 && rows_by(p->x, p->x_st, a->T, a->x_dtype, 16) &&
                 rows_by(p->dt, p->dt_st, a->T, a->dt_dtype, 16) && (ds == es || per * ds % 16 == 0) && rows_by(p->z, p->z_st, a->T, a->x_dtype, 16);
  p->fast_vectors = a->S * es % 16 == 0 && rows_by(p->B, p->B_st, a->T, a->x_dtype, 16) && rows_by(p->Cm, p->C_st, a->T, a->x_dtype, 16) &&
                    p->B_sg * es % 16 == 0 && p->C_sg * es % 16 == 0;
  p->quad_vectors = a->S % 4 == 0 && aligned(a->A, 16) && rows_by(p->B, p->B_st, a->T, a->x_dtype, 4 * es) &&
                    rows_by(p->Cm, p->C_st, a->T, a->x_dtype, 4 * es) && p->B_sg % 4 == 0 && p->C_sg % 4 == 0;
  p->pair_out = a->C % 2 == 0 && per % 2 == 0;
  return GDP_OK;
}

// Outputs against the inputs that `common` has resolved, and d_output (`dy`) in the backward pass.
gdp_status scan_apart(const SsmProblem &p, int type, std::initializer_list<Span> outs, const Span &dy) {
  const int dt_type = p.dt_f32 ? GDP_DTYPE_F32 : type;
  return apart_ok(p.p.T, outs,
                  {rows(p.x, p.x_st, p.C, type, "x"), rows(p.dt, p.dt_st, p.C, dt_type, "dt"), rows(p.z, p.z_st, p.C, type, "z"),
                   Span{p.B, p.B_st, p.S, type, "B", p.G, p.B_sg}, Span{p.Cm, p.C_st, p.S, type, "C", p.G, p.C_sg}, dy});
}

gdp_status resolve(const gdp_scan_args *a, bool step, SsmProblem *p) {
  set_last_error("");
  if (!a) return fail(GDP_ERR_INVALID_ARG, "args is NULL");
  gdp_status st = common(a, p);
  if (st != GDP_OK) return st;
  if (step && a->T != a->N) return fail(GDP_ERR_INVALID_ARG, "decode takes one token per sequence: T == N");
  if ((st = rows_ok(a->output, a->C, a->T, a->C, a->x_dtype, "output")) != GDP_OK) return st;
  if (!step && !a->cu_seqlens) return fail(GDP_ERR_INVALID_ARG, "cu_seqlens is required");
  if ((st = states_ok(a->initial_state, a->output_state, a->state, a->state_indices, a->num_slots, 4,
                      sizeof(float) * (size_t)a->N * (size_t)a->C * (size_t)a->S)) != GDP_OK)
    return st;
  if (!aligned(a->chunk_states, 4)) return fail(GDP_ERR_INVALID_ARG, "state buffers must be aligned to their elements");
  if ((st = scan_apart(*p, a->x_dtype, {dense(a->output, a->C, a->x_dtype, "output")}, Span{})) != GDP_OK) return st;
  p->y = a->output;
  p->s = StateModes{a->initial_state, a->output_state, a->state, a->state_indices, a->num_slots};
  p->chunks = step ? nullptr : a->chunk_states;
  p->pair_out = p->pair_out && aligned(a->output, 2 * dtype_size(a->x_dtype));
  p->zero_pad = !step && a->zero_padding != 0;
  p->quad_states = a->S % 4 == 0 && aligned(a->initial_state, 16) && aligned(a->output_state, 16) && aligned(a->state, 16) && aligned(a->chunk_states, 16);
  return GDP_OK;
}

bool scan_shape(int64_t T, int64_t N, int64_t C, int64_t S, int64_t G) {
  return T >= 0 && N >= 0 && C >= 1 && S >= 1 && S <= 64 && G >= 1 && C % G == 0 && C <= (1 << 20) && T <= INT32_MAX && N < INT32_MAX;
}
int64_t enter_bytes(int64_t pieces, int64_t C, int64_t S) { return (pieces * C * S * 4 + 255) / 256 * 256; }
int64_t over_rows_bytes(int64_t workers, int64_t C, int64_t S) { return (workers * ssm_sum_cols(C, S) * 4 + 255) / 256 * 256; }

}  // namespace
}  // namespace layer
}  // namespace gdp

GDP_EXPORT size_t gdp_scan_forward_workspace_bytes(int64_t T, int64_t N, int64_t C, int64_t S, int64_t G) {
  using namespace gdp::layer;
  if (!scan_shape(T, N, C, S, G)) return 0;
  const int64_t piece = ssm_piece(T, N, G * ssm_tiles(C / G, S), sm_count(), kSsmForward);
  return piece ? (size_t)enter_bytes(T / piece + N, C, S) + (size_t)(T / piece + N) * (size_t)C * 4 : 0;
}

GDP_EXPORT gdp_status gdp_selective_scan(const gdp_scan_args *args, void *stream) {
  using namespace gdp::layer;
  SsmProblem p;
  const gdp_status st = resolve(args, false, &p);
  if (st != GDP_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  if (p.p.N == 0) return p.zero_pad ? zero_out(p.y, (size_t)(p.p.T * p.C), args->x_dtype, s) : GDP_OK;
  const size_t need = gdp_scan_forward_workspace_bytes(args->T, args->N, args->C, args->S, args->G);
  if (need && (!args->workspace || !aligned(args->workspace, 256) || args->workspace_bytes < need))
    return fail(GDP_ERR_WORKSPACE, "workspace missing, not 256-byte aligned or smaller than gdp_scan_forward_workspace_bytes");
  p.piece = ssm_piece(p.p.T, p.p.N, p.G * p.tiles, p.sms, kSsmForward);
  p.pieces = p.piece ? p.p.T / p.piece + p.p.N : p.p.N;
  p.ranked = !p.piece && ssm_ranked(p.p.T, p.p.N, p.G * p.tiles, p.sms);
  if (p.piece) {
    p.enter = static_cast<float *>(args->workspace);
    p.spans = p.enter + enter_bytes(p.pieces, p.C, p.S) / 4;
  }
  return cuda_status(args->x_dtype == GDP_DTYPE_BF16  ? launch_ssm_fwd<__nv_bfloat16>(p, s)
                     : args->x_dtype == GDP_DTYPE_F16 ? launch_ssm_fwd<__half>(p, s)
                                                      : launch_ssm_fwd<float>(p, s),
                     "selective scan kernel");
}

GDP_EXPORT gdp_status gdp_selective_scan_decode(const gdp_scan_args *args, void *stream) {
  using namespace gdp::layer;
  SsmProblem p;
  const gdp_status st = resolve(args, true, &p);
  if (st != GDP_OK || p.p.N == 0) return st;
  cudaStream_t s = (cudaStream_t)stream;
  return cuda_status(args->x_dtype == GDP_DTYPE_BF16  ? launch_ssm_step<__nv_bfloat16>(p, s)
                     : args->x_dtype == GDP_DTYPE_F16 ? launch_ssm_step<__half>(p, s)
                                                      : launch_ssm_step<float>(p, s),
                     "selective scan step kernel");
}

GDP_EXPORT int64_t gdp_scan_chunk_rows(int64_t T, int64_t N) { return T < 0 || N < 0 ? 0 : T / GDP_SCAN_CHUNK + N; }

GDP_EXPORT size_t gdp_scan_workspace_bytes(int64_t T, int64_t N, int64_t C, int64_t S, int64_t G) {
  using namespace gdp::layer;
  if (!scan_shape(T, N, C, S, G)) return 0;
  const int64_t tiles = G * ssm_tiles(C / G, S), piece = ssm_piece(T, N, tiles, sm_count(), kSsmBackward), pieces = piece ? T / piece + N : N;
  size_t bytes = (size_t)over_rows_bytes(ssm_workers(pieces, tiles, sm_count()), C, S) + (size_t)tiles * (size_t)T * (size_t)(8 * 4 * ssm_lanes(S));
  if (piece) bytes += (size_t)enter_bytes(pieces, C, S) + (size_t)pieces * (size_t)C * 4;
  return bytes;
}

GDP_EXPORT gdp_status gdp_selective_scan_backward(const gdp_scan_backward_args *a, void *stream) {
  using namespace gdp::layer;
  gdp::set_last_error("");
  if (!a) return fail(GDP_ERR_INVALID_ARG, "args is NULL");
  SsmProblem p;
  gdp_status st = common(a, &p);
  if (st != GDP_OK) return st;
  if ((st = rows_ok(a->d_output, a->d_output_stride_t, a->T, a->C, a->x_dtype, "d_output")) != GDP_OK) return st;
  if ((st = rows_ok(a->dx, a->C, a->T, a->C, a->x_dtype, "dx")) != GDP_OK) return st;
  if ((st = rows_ok(a->ddt, a->C, a->T, a->C, a->dt_dtype, "ddt")) != GDP_OK) return st;
  if ((st = rows_ok(a->dB, a->S, a->T, a->S, a->x_dtype, "dB")) != GDP_OK) return st;
  if ((st = rows_ok(a->dC, a->S, a->T, a->S, a->x_dtype, "dC")) != GDP_OK) return st;
  if (a->z && (st = rows_ok(a->dz, a->C, a->T, a->C, a->x_dtype, "dz")) != GDP_OK) return st;
  if (!a->cu_seqlens) return fail(GDP_ERR_INVALID_ARG, "cu_seqlens is required");
  if (!a->dA || (a->D != nullptr) != (a->dD != nullptr) || (a->dt_bias != nullptr) != (a->ddt_bias != nullptr))
    return fail(GDP_ERR_INVALID_ARG, "dA is required, dD goes with D and ddt_bias with dt_bias");
  if (a->T > 0 && a->N > 0 && !a->chunk_states) return fail(GDP_ERR_INVALID_ARG, "chunk_states is required");
  if (!aligned(a->chunk_states, 4) || !aligned(a->d_final_state, 4) || !aligned(a->d_initial_state, 4) || !aligned(a->dA, 4) || !aligned(a->dD, 4) ||
      !aligned(a->ddt_bias, 4))
    return fail(GDP_ERR_INVALID_ARG, "fp32 buffers must be 4-byte aligned");
  const size_t state_bytes = sizeof(float) * (size_t)a->N * (size_t)a->C * (size_t)a->S;
  if (overlap(a->d_final_state, a->d_initial_state, state_bytes)) return fail(GDP_ERR_ALIAS, "d_initial_state overlaps d_final_state");
  if (!a->workspace || !aligned(a->workspace, 256) || a->workspace_bytes < gdp_scan_workspace_bytes(a->T, a->N, a->C, a->S, a->G))
    return fail(GDP_ERR_WORKSPACE, "workspace missing, not 256-byte aligned or smaller than gdp_scan_workspace_bytes");
  const int type = a->x_dtype;
  const int64_t vectors = a->G * a->S;
  if ((st = scan_apart(p, type,
                       {dense(a->dx, a->C, type, "dx"), dense(a->ddt, a->C, a->dt_dtype, "ddt"), dense(a->z ? a->dz : nullptr, a->C, type, "dz"),
                        dense(a->dB, vectors, type, "dB"), dense(a->dC, vectors, type, "dC")},
                       rows(a->d_output, stride_of(a->d_output_stride_t, a->T, a->C), a->C, type, "d_output"))) != GDP_OK)
    return st;
  cudaStream_t s = (cudaStream_t)stream;
  if (a->N == 0) {  // every row is padding
    const size_t rows = (size_t)(a->T * a->C), vectors = (size_t)(a->T * a->G * a->S);
    if ((st = zero_out(a->dx, rows, a->x_dtype, s)) != GDP_OK || (st = zero_out(a->ddt, rows, a->dt_dtype, s)) != GDP_OK ||
        (st = zero_out(a->z ? a->dz : nullptr, rows, a->x_dtype, s)) != GDP_OK || (st = zero_out(a->dB, vectors, a->x_dtype, s)) != GDP_OK ||
        (st = zero_out(a->dC, vectors, a->x_dtype, s)) != GDP_OK || (st = zero_out(a->dA, (size_t)(a->C * a->S), GDP_DTYPE_F32, s)) != GDP_OK ||
        (st = zero_out(a->dD, (size_t)a->C, GDP_DTYPE_F32, s)) != GDP_OK)
      return st;
    return zero_out(a->ddt_bias, (size_t)a->C, GDP_DTYPE_F32, s);
  }
  p.dy = a->d_output; p.dy_st = stride_of(a->d_output_stride_t, a->T, a->C);
  p.dfin = a->d_final_state;
  p.chunks = const_cast<float *>(a->chunk_states);
  p.dx = a->dx; p.ddt = a->ddt; p.dz = a->z ? a->dz : nullptr; p.dB = a->dB; p.dC = a->dC; p.dinit = a->d_initial_state;
  p.quad_states = a->S % 4 == 0 && aligned(a->chunk_states, 16) && aligned(a->d_final_state, 16) && aligned(a->d_initial_state, 16);
  p.fast_rows = p.fast_rows && rows_by(p.dy, p.dy_st, p.p.T, a->x_dtype, 16);
  p.pair_out = p.pair_out && aligned(p.dx, 2 * dtype_size(a->x_dtype)) && aligned(p.dz, 2 * dtype_size(a->x_dtype)) && aligned(p.ddt, 2 * dtype_size(a->dt_dtype));
  p.piece = ssm_piece(p.p.T, p.p.N, p.G * p.tiles, p.sms, kSsmBackward);
  p.pieces = p.piece ? p.p.T / p.piece + p.p.N : p.p.N;
  p.ranked = !p.piece && ssm_ranked(p.p.T, p.p.N, p.G * p.tiles, p.sms);
  p.workers = ssm_workers(p.pieces, p.G * p.tiles, p.sms);
  p.over_rows = static_cast<float *>(a->workspace);
  p.over_channels = p.over_rows + over_rows_bytes(p.workers, p.C, p.S) / 4;
  if (p.piece) {
    p.enter = p.over_channels + p.G * p.tiles * p.p.T * 8 * ssm_lanes(p.S);
    p.spans = p.enter + enter_bytes(p.pieces, p.C, p.S) / 4;
  }
  cudaError_t e = a->x_dtype == GDP_DTYPE_BF16  ? launch_ssm_bwd<__nv_bfloat16>(p, s)
                  : a->x_dtype == GDP_DTYPE_F16 ? launch_ssm_bwd<__half>(p, s)
                                                : launch_ssm_bwd<float>(p, s);
  if (e == cudaSuccess) {
    ColumnSums c{};
    c.from = p.over_rows; c.parts = p.workers; c.cols = ssm_sum_cols(p.C, p.S);
    c.to[0] = a->dA; c.to[1] = a->dD; c.to[2] = a->ddt_bias;
    c.first[1] = p.C * p.S; c.first[2] = p.C * (p.S + 1); c.first[3] = p.C * (p.S + 2);
    e = launch_column_sums(c, s);
  }
  return cuda_status(e, "selective scan backward kernels");
}
