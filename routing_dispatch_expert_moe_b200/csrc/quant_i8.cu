// Rows to 8-bit integers with one scale each, optionally dispatched to their experts.
//
// Handbook digest (agihunt.info), "已确认", bullet "量化与推理" (routed experts kept in few bits);
// handbook news post (hub.geekagi.cn), "MoE 到底省了什么" (sending each token to its experts).
//
//   f = 127 (1 / amax) in fp32, both steps rounded; q = rint(x f) to the nearest even;
//   scale = amax / 127
// A row of zeros, or one whose amax is below 2^-120 (f would overflow below 2^-121),
// gives q = 0 and scale 0.  A row with an infinity or a NaN gives q = 0 and a
// NaN scale, so exactly the products of that row are NaN.
//
// Bound by HBM: it reads a row once (2 or 4 bytes an element), keeps it in registers between
// the maximum and the rounding, and writes one byte an element, or one to each of the k kept
// rows of x_perm (dispatch of 8-bit rows moves half the bytes of a bf16 permute).  A row is
// given TPR threads, 16 elements each at a time, so that its loads are all in flight at once.
// 65,536 bf16 rows of 2048: 74 us, 5.4 TB/s (the bytes need 61).
#include "common.cuh"
#include "row8.cuh"

namespace moe {
namespace {

constexpr int kQThreads = 256;
constexpr uint32_t kTiny = (127u - 120u) << 23;            // the bits of 2^-120
constexpr unsigned kFull = 0xffffffffu;

template <typename T>
struct Row16;
template <>
struct Row16<__nv_bfloat16> {
  uint4 a, b;
  __device__ __forceinline__ void load(const void* base, long long e) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + e);
    a = ld_stream(p);
    b = ld_stream(p + 1);
  }
  __device__ __forceinline__ void get(float* f) const {
    unpack8(a, f);
    unpack8(b, f + 8);
  }
};
template <>
struct Row16<float> {
  uint4 a[4];
  __device__ __forceinline__ void load(const void* base, long long e) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + e);
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = ld_stream(p + i);
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[4 * i] = __uint_as_float(a[i].x);
      f[4 * i + 1] = __uint_as_float(a[i].y);
      f[4 * i + 2] = __uint_as_float(a[i].z);
      f[4 * i + 3] = __uint_as_float(a[i].w);
    }
  }
};

// Four rounded values as packed bytes (|x f| <= 127 (1 + 2^-23): the cast needs no clamp).
__device__ __forceinline__ uint32_t pack_i8(const float* x, float f) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) r |= ((uint32_t)__float2int_rn(x[i] * f) & 0xffu) << (8 * i);
  return r;
}

// |x| as ordered bits: NaN above infinity above every number, so one maximum finds them.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// TPR threads a row (a power of two), V groups of 16 elements a thread.  DISPATCH: the rows
// row_of[t, 0 .. k) take the token's bytes and its scale; otherwise row t does.
template <typename InT, int TPR, int V, bool DISPATCH>
__global__ void __launch_bounds__(kQThreads)
quantize_rows_kernel(const void* __restrict__ x, long long rows, int cols, const int32_t* __restrict__ row_of, int k,
                     long long rows_max, int8_t* __restrict__ q, float* __restrict__ scale, int* err) {
  constexpr int RPB = kQThreads / TPR;                     // rows a block has at a time
  __shared__ uint32_t s_max[2][kQThreads / 32];
  const int tr = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int n16 = cols / 16;
  const long long passes = (rows + RPB - 1) / RPB;
  int buf = 0;
  for (long long it = blockIdx.x; it < passes; it += gridDim.x) {
    const long long r = it * RPB + sub;
    const bool row = r < rows;
    Row16<InT> in[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (row && tr + v * TPR < n16) in[v].load(x, r * cols + (tr + v * TPR) * 16);
    uint32_t m = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!(row && tr + v * TPR < n16)) continue;
      float f[16];
      in[v].get(f);
#pragma unroll
      for (int i = 0; i < 16; ++i) m = max(m, abs_bits(f[i]));
    }
    m = __reduce_max_sync(kFull, m);
    if constexpr (TPR > 32) {
      const int wp = threadIdx.x >> 5;
      if ((threadIdx.x & 31) == 0) s_max[buf][wp] = m;
      __syncthreads();                                     // two buffers: one barrier a pass
      constexpr int WPR = TPR / 32;
      const int w0 = wp / WPR * WPR;
#pragma unroll
      for (int i = 0; i < WPR; ++i) m = max(m, s_max[buf][w0 + i]);
      buf ^= 1;
    }
    if (!row) continue;
    const bool fine = m < 0x7f800000u;
    const float amax = __uint_as_float(m);
    const bool some = m >= kTiny;
    const float f = fine && some ? 127.f * (1.f / amax) : 0.f;
    const float sc = !fine ? __uint_as_float(0x7fc00000u) : some ? amax / 127.f : 0.f;
    uint4 o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      o[v] = make_uint4(0, 0, 0, 0);
      if (!fine || !(tr + v * TPR < n16)) continue;
      float e[16];
      in[v].get(e);
      o[v] = make_uint4(pack_i8(e, f), pack_i8(e + 4, f), pack_i8(e + 8, f), pack_i8(e + 12, f));
    }
    for (int j = 0; j < (DISPATCH ? k : 1); ++j) {
      long long to = r;
      if constexpr (DISPATCH) {
        to = __ldg(row_of + r * k + j);
        if (to >= rows_max) { record_error(err, MOE_DEVERR_ROW); continue; }
        if (to < 0) continue;
      }
      if (tr == 0) scale[to] = sc;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (tr + v * TPR < n16) *reinterpret_cast<uint4*>(q + to * cols + (tr + v * TPR) * 16) = o[v];
    }
  }
}

template <typename InT, int TPR, int V>
moe_status run_quantize(const void* x, long long rows, int cols, const int32_t* row_of, int k, long long rows_max,
                        int8_t* q, float* scale, cudaStream_t s) {
  constexpr int RPB = kQThreads / TPR;
  long long blocks = (rows + RPB - 1) / RPB;
  const long long cap = (long long)num_sms() * 16;
  if (blocks > cap) blocks = cap;
  if (row_of)
    quantize_rows_kernel<InT, TPR, V, true><<<(unsigned)blocks, kQThreads, 0, s>>>(x, rows, cols, row_of, k, rows_max,
                                                                                  q, scale, err_ptr());
  else
    quantize_rows_kernel<InT, TPR, V, false><<<(unsigned)blocks, kQThreads, 0, s>>>(x, rows, cols, row_of, k,
                                                                                   rows_max, q, scale, err_ptr());
  return check_launch();
}

// One group of 16 a thread up to 4096 elements, then two and four.
template <typename InT>
moe_status quantize(const void* x, long long rows, int cols, const int32_t* row_of, int k, long long rows_max,
                    int8_t* q, float* scale, cudaStream_t s) {
  const int n16 = cols / 16;
#define MOE_Q(TPR, V) return run_quantize<InT, TPR, V>(x, rows, cols, row_of, k, rows_max, q, scale, s)
  if (n16 <= 32) MOE_Q(32, 1);
  if (n16 <= 64) MOE_Q(64, 1);
  if (n16 <= 128) MOE_Q(128, 1);
  if (n16 <= 256) MOE_Q(256, 1);
  if (n16 <= 512) MOE_Q(256, 2);
  MOE_Q(256, 4);
#undef MOE_Q
}

}  // namespace

moe_status launch_quantize_rows_i8(const void* x, int dtype, long long rows, int cols, const int32_t* row_of, int k,
                                   long long rows_max, int8_t* q, float* scale, cudaStream_t s) {
  if (dtype == MOE_F32) return quantize<float>(x, rows, cols, row_of, k, rows_max, q, scale, s);
  return quantize<__nv_bfloat16>(x, rows, cols, row_of, k, rows_max, q, scale, s);
}

}  // namespace moe
