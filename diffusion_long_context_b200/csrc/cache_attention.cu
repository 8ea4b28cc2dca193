// Attention of few queries over the 8-bit paged cache (first form: one CTA per query row).
#include <algorithm>

#include "cache.cuh"

namespace focus {
namespace {

struct CacheAttnArgs {
  const __nv_bfloat16* Q;
  const int32_t* n_q;
  const uint8_t* code[2];
  const float* scale[2];
  const int32_t* table;
  const int32_t* lens;       // dense
  const int32_t* P;          // sparse
  const int32_t* g0;
  const int32_t* sinks;
  const int32_t* blocks;
  __nv_bfloat16* O;
  int table_cols, n_pages, page, B, Hq, Hkv, qcap, G, S, C;
  float scale_log2;
  int* dev_err;
};

// Position of key slot j of (b, h), or -1: [current block | kept blocks | sinks].
__device__ int slot_position(const CacheAttnArgs& a, int b, int h, int j) {
  const int g0 = a.g0[b], P = a.P[b];
  if (j < a.G) return g0 + j;
  j -= a.G;
  const int32_t* blk = a.blocks + (static_cast<size_t>(b) * a.Hkv + h) * a.C;
  if (j < a.C * a.page) {
    const int v = blk[j / a.page];
    for (int i = 0; i < j / a.page; ++i)
      if (blk[i] == v) return -1;
    const int pos = v * a.page + j % a.page;
    return v >= 0 && pos < P && !(pos >= g0 && pos < g0 + a.G) ? pos : -1;
  }
  j -= a.C * a.page;
  const int32_t* snk = a.sinks + (static_cast<size_t>(b) * a.Hkv + h) * a.S;
  const int pos = snk[j];
  if (pos < 0 || (pos >= g0 && pos < g0 + a.G)) return -1;
  for (int i = 0; i < j; ++i)
    if (snk[i] == pos) return -1;
  if (pos < P)
    for (int i = 0; i < a.C; ++i)
      if (blk[i] == pos / a.page) return -1;
  return pos;
}

template <int FMT, int D, bool SPARSE>
__global__ void __launch_bounds__(128) cache_attn_rows_kernel(const CacheAttnArgs a) {
  constexpr int N = D / 32;
  __shared__ float s_o[4][D], s_m[4], s_l[4];
  griddep_wait();
  griddep_launch_dependents();
  const int row = blockIdx.x, i = row % a.qcap, hq = row / a.qcap % a.Hq, b = row / (a.qcap * a.Hq);
  const int h = hq / (a.Hq / a.Hkv), warp = warp_id(), lane = lane_id();
  __nv_bfloat16* O = a.O + static_cast<size_t>(row) * D;
  float q[N], o[N], m = -INFINITY, l = 0.f;
  for (int j = 0; j < N; ++j) {
    q[j] = __bfloat162float(a.Q[static_cast<size_t>(row) * D + lane * N + j]) * a.scale_log2;
    o[j] = 0.f;
  }
  int n = SPARSE ? a.G + a.C * a.page + a.S : max(0, min(a.lens[b], a.table_cols * a.page));
  if (a.n_q && i >= a.n_q[b]) n = 0;
  for (int s = warp; s < n; s += 4) {
    const int pos = SPARSE ? slot_position(a, b, h, s) : s;
    if (pos < 0) continue;
    const int page = checked_page(a.table, a.table_cols, b, pos / a.page, a.n_pages, a.dev_err);
    if (page < 0) continue;
    const size_t ph = static_cast<size_t>(page) * a.Hkv + h;
    const size_t off = (ph * a.page + pos % a.page) * D + lane * N;
    float k[4], v[4];
    uint32_t wk, wv;
    if (N == 4) {
      wk = *reinterpret_cast<const uint32_t*>(a.code[0] + off);
      wv = *reinterpret_cast<const uint32_t*>(a.code[1] + off);
    } else {
      wk = *reinterpret_cast<const uint16_t*>(a.code[0] + off);
      wv = *reinterpret_cast<const uint16_t*>(a.code[1] + off);
    }
    decode4<FMT>(wk, k);
    decode4<FMT>(wv, v);
    float t = 0.f;
    for (int j = 0; j < N; ++j) t += q[j] * k[j];
    for (int x = 16; x; x >>= 1) t += __shfl_xor_sync(0xffffffffu, t, x);
    t *= a.scale[0][ph];
    const float mn = fmaxf(m, t), c = exp2f(m - mn), p = exp2f(t - mn), pv = p * a.scale[1][ph];
    l = l * c + p;
    for (int j = 0; j < N; ++j) o[j] = o[j] * c + pv * v[j];
    m = mn;
  }
  for (int j = 0; j < N; ++j) s_o[warp][lane * N + j] = o[j];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  const float M = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  if (threadIdx.x < D) {
    float x = 0.f, L = 0.f;
    for (int w = 0; w < 4; ++w) {
      const float c = s_l[w] == 0.f ? 0.f : exp2f(s_m[w] - M);
      x += c * s_o[w][threadIdx.x];
      L += c * s_l[w];
    }
    O[threadIdx.x] = __float2bfloat16_rn(L == 0.f ? 0.f : x / L);
  }
}

int run_cache_attention(const CacheAttnArgs& a, int format, int d, bool sparse, cudaStream_t stream) {
  const long long rows = static_cast<long long>(a.B) * a.Hq * a.qcap;
  if (rows == 0) return FOCUS_OK;
  FOCUS_CHECK_ARG(rows < (1LL << 31), "too large");
  void (*kern)(const CacheAttnArgs);
  if (format == FOCUS_CACHE_E4M3)
    kern = d == 128 ? (sparse ? cache_attn_rows_kernel<0, 128, true> : cache_attn_rows_kernel<0, 128, false>)
                    : (sparse ? cache_attn_rows_kernel<0, 64, true> : cache_attn_rows_kernel<0, 64, false>);
  else
    kern = d == 128 ? (sparse ? cache_attn_rows_kernel<1, 128, true> : cache_attn_rows_kernel<1, 128, false>)
                    : (sparse ? cache_attn_rows_kernel<1, 64, true> : cache_attn_rows_kernel<1, 64, false>);
  const cudaError_t e = launch_k(kern, dim3(static_cast<unsigned>(rows)), dim3(128), 0, stream, a);
  note_launch();
  if (e != cudaSuccess) {
    cudaGetLastError();
    set_error("cache attention launch: %s", cudaGetErrorString(e));
    return FOCUS_ERR_CUDA;
  }
  return FOCUS_OK;
}

int check_attention(const focus_bf16* Q, const focus_cache* cache, const int32_t* table, int table_cols, int B, int Hq,
                    int qcap, const focus_bf16* O, const void* ws, size_t ws_bytes) {
  FOCUS_CHECK_ARG(Q && O, "null pointer argument");
  if (const int st = check_cache(cache, table, table_cols, true)) return st;
  FOCUS_CHECK_ARG(B >= 0 && Hq >= 1 && qcap >= 1, "bad sizes (B=%d Hq=%d qcap=%d)", B, Hq, qcap);
  FOCUS_CHECK_ARG(Hq % cache->Hkv == 0, "Hq %d is not a multiple of Hkv %d", Hq, cache->Hkv);
  FOCUS_CHECK_ARG(aligned16(Q) && aligned16(O), "tensors must be 16-byte aligned");
  FOCUS_CHECK_ARG(static_cast<long long>(table_cols) * cache->page < (1LL << 31), "table of 2^31 positions or more");
  const size_t need = focus_cache_workspace_bytes(B, Hq, cache->Hkv, cache->d, qcap);
  if (need) {
    FOCUS_CHECK_ARG(ws, "null workspace (%zu bytes needed)", need);
    FOCUS_CHECK_ARG((reinterpret_cast<uintptr_t>(ws) & 255u) == 0, "workspace must be 256-byte aligned");
    if (ws_bytes < need) {
      set_error("workspace of %zu bytes, %zu needed", ws_bytes, need);
      return FOCUS_ERR_CAPACITY;
    }
  }
  return FOCUS_OK;
}

CacheAttnArgs attn_args(const focus_bf16* Q, const int32_t* n_q, const focus_cache* c, const int32_t* table,
                        int table_cols, int B, int Hq, int qcap, float scale, focus_bf16* O) {
  CacheAttnArgs a{};
  a.Q = reinterpret_cast<const __nv_bfloat16*>(Q);
  a.n_q = n_q;
  a.code[0] = static_cast<const uint8_t*>(c->k);
  a.code[1] = static_cast<const uint8_t*>(c->v);
  a.scale[0] = c->k_scale;
  a.scale[1] = c->v_scale;
  a.table = table;
  a.table_cols = table_cols;
  a.n_pages = c->n_pages;
  a.page = c->page;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = c->Hkv;
  a.qcap = qcap;
  a.O = reinterpret_cast<__nv_bfloat16*>(O);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.dev_err = device_error_word();
  return a;
}

}  // namespace
}  // namespace focus

using namespace focus;

extern "C" size_t focus_cache_workspace_bytes(int, int, int, int, int) { return 0; }

extern "C" int focus_cache_attention(const focus_bf16* Q, const int32_t* n_q, const focus_cache* cache,
                                     const int32_t* table, int table_cols, const int32_t* lens, int B, int Hq,
                                     int qcap, float scale, focus_bf16* O, void* ws, size_t ws_bytes, void* stream) {
  if (const int st = check_attention(Q, cache, table, table_cols, B, Hq, qcap, O, ws, ws_bytes)) return st;
  FOCUS_CHECK_ARG(lens, "null pointer argument");
  CacheAttnArgs a = attn_args(Q, n_q, cache, table, table_cols, B, Hq, qcap, scale, O);
  a.lens = lens;
  return run_cache_attention(a, cache->format, cache->d, false, static_cast<cudaStream_t>(stream));
}

extern "C" int focus_cache_sparse_attention(const focus_bf16* Q_active, const int32_t* n_active,
                                            const focus_cache* cache, const int32_t* table, int table_cols,
                                            const int32_t* P, const int32_t* g0, int G, const int32_t* sinks, int S,
                                            const int32_t* blocks, int C, int B, int Hq, int qcap, float scale,
                                            focus_bf16* O_active, void* ws, size_t ws_bytes, void* stream) {
  if (const int st = check_attention(Q_active, cache, table, table_cols, B, Hq, qcap, O_active, ws, ws_bytes)) return st;
  FOCUS_CHECK_ARG(P && g0 && blocks && (S == 0 || sinks), "null pointer argument");
  FOCUS_CHECK_ARG(G >= 1 && S >= 0 && C >= 1, "bad sizes (G=%d S=%d C=%d)", G, S, C);
  if (S > 1024 || C > 1024) {
    set_error("cache sparse attention: S and C up to 1024 (got %d and %d)", S, C);
    return FOCUS_ERR_UNSUPPORTED;
  }
  CacheAttnArgs a = attn_args(Q_active, n_active, cache, table, table_cols, B, Hq, qcap, scale, O_active);
  a.P = P;
  a.g0 = g0;
  a.G = G;
  a.sinks = sinks;
  a.S = S;
  a.blocks = blocks;
  a.C = C;
  return run_cache_attention(a, cache->format, cache->d, true, static_cast<cudaStream_t>(stream));
}
