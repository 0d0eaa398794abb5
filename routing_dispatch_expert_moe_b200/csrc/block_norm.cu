// The norms around a block, fused with its gate, the residual and its scale, forward and
// backward; forward also with the combine of the block's expert rows in front.
//
// "Hugging Face 图解 Mixture of Experts（MoE）原理、训练与推理权衡", section "什么是混合专家模型"
// (the MoE layer stands in a transformer block between its norm and the residual add) and
// section "什么是稀疏性？", eq. y = sum_i G(x)_i E_i(x).
//
//   b  = y                          or  w_post * y / rms(y),   rms(y) = sqrt(mean y^2 + eps)
//   x' = alpha r + gate * b
//   n  = w_pre * x' / rms(x')
// with u = dL/dx' (u = d_x + the pre-norm's part) the gradients are
//   u      = d_x + (g - xh mean(g xh)) / rms(x'),  g = w_pre d_n,  xh = x' / rms(x')
//   d_r    = alpha u;      d_w_pre = sum_t d_n xh
//   d_gate = sum_t u b;    d_w_post = sum_t u gate yh,   yh = y / rms(y)
//   d_y    = (h - yh mean(h yh)) / rms(y),  h = u gate w_post      (u gate without a post-norm)
//
// Bound by HBM: each input is read once and each output written once, the row between them in
// registers.  A block has a row; a thread has V vectors of eight neighbouring elements.  Sums are
// fp32: a thread's elements, a shuffle, then the warps' sums through shared memory.  Forward with
// the combine, 8192 tokens, d = 2048, k = 8: 72 us where the bytes need 54 (85 with a grid of
// persistent blocks).
// The backward pass gives each block a run of rows; it keeps the column sums in registers over
// the rows of a gate group (the gate's and the post-norm weight's are one sum, sum_t u yh, times
// the other's value) and over all its rows (the pre-norm weight's), and a second kernel adds the
// blocks' partial sums in a fixed order (results repeat bit for bit).  8192 tokens, d = 2048:
// 47 us with the sums, where the bytes need 31: two block-wide sums a row, half the issue rate.
// 4096 tokens, d = 7168, fp32 residual: 104 us (110 with pre read through the first-level cache),
// where the bytes need 81.  Where shared memory holds one row's inputs only, its loads wait for the
// row before: fp32 residual, 8192 x 2048 67 us (46), 4096 x 4096 70 (46), 4096 x 8192 135 (92); all
// fp32 82 (61), 90 (61) and 178 (123).
#include "common.cuh"
#include "f32x2.cuh"
#include "tc_prims.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kNormMaxWarps = 16;

// Sums over the block; `part` is this call's own slice of shared memory, so that a row needs one
// barrier for each reduction.  Every warp adds the warps' sums itself (at most 16: four steps).
__device__ __forceinline__ float block_sum(float a, float* part, int warps) {
#pragma unroll
  for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(kFull, a, o);
  if (warps == 1) return a;
  const int lane = threadIdx.x & 31;
  if (lane == 0) part[threadIdx.x >> 5] = a;
  __syncthreads();
  a = (lane & 15) < warps ? part[lane & 15] : 0.f;
#pragma unroll
  for (int o = 8; o; o >>= 1) a += __shfl_xor_sync(kFull, a, o);
  return a;
}
__device__ __forceinline__ float2 block_sum2(float a, float b, float2* part, int warps) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(kFull, a, o);
    b += __shfl_xor_sync(kFull, b, o);
  }
  if (warps == 1) return make_float2(a, b);
  const int lane = threadIdx.x & 31;
  if (lane == 0) part[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  float2 s = (lane & 15) < warps ? part[lane & 15] : make_float2(0.f, 0.f);
#pragma unroll
  for (int o = 8; o; o >>= 1) {
    s.x += __shfl_xor_sync(kFull, s.x, o);
    s.y += __shfl_xor_sync(kFull, s.y, o);
  }
  return s;
}
// 1 / rms from a row's sum of squares (rsqrtf: within 2 steps).
__device__ __forceinline__ float inv_rms(float ss, float inv_d, float eps) { return rsqrtf(fmaf(ss, inv_d, eps)); }

// Eight elements of a row in its storage type, as loaded; `oct` makes them pairs of fp32.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const void* base, long long e) {
    a = ld_stream(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + e));
  }
  __device__ __forceinline__ Oct oct() const { return oct_bf16(a); }
};
template <>
struct Raw8<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const void* base, long long e) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + e);
    a = ld_stream(p);
    b = ld_stream(p + 1);
  }
  __device__ __forceinline__ Oct oct() const { return oct_f32(a, b); }
};
// Eight of a parameter's values, or ones where it is not given.
__device__ __forceinline__ Oct param8(const float* p, long long e) {
  if (!p) return oct_const(1.f);
  const uint4* q = reinterpret_cast<const uint4*>(p + e);
  return oct_f32(__ldg(q), __ldg(q + 1));
}

struct NormArgs {
  const void* r;              // [T, d]
  const void* y;              // [T, d], or the expert rows [rows_max, d], or null
  const float* post;          // [d] or null
  const float* gate;          // [G, d] or null
  const float* pre;           // [d] or null
  const int32_t* row_of;      // combine: [T, k]
  const float* topk_gate;     // combine: [T, k] or null
  const void* shared_y;       // combine: [T, d] or null
  void* y_out;                // combine: [T, d] or null
  void* x_out;                // [T, d] or null
  void* n_out;                // [T, d] or null
  long long rows_max;
  float alpha, eps, inv_d;    // inv_d = 1 / d
  int T, d, per_gate, k;      // per_gate: tokens that share a gate row
  int* err;
};

// YT: y or the expert rows; RT: the residual stream; NT: the normed rows.
// V = 1: five blocks, 51 registers; fp32 expert rows (32 bytes a load, four in flight) spill some of
// them (84 to 100 bytes): 8192 tokens, d = 2048, k = 8, 116 us where the bytes need 97, as near as the
// bf16 rows' 68 to 56.
template <typename YT, typename RT, typename NT, int V, bool COMBINE>
__global__ void __launch_bounds__(V == 1 ? 256 : 512, V == 1 ? 5 : 1)
block_norm_kernel(const NormArgs a) {
  __shared__ float part[2][kNormMaxWarps];
  const int warps = blockDim.x >> 5;
  const int n8 = a.d >> 3;
  const long long t = blockIdx.x;
  // the token's rows and gates, slot j's in lane j of every warp
  int my_row = -1;
  float my_gate = 1.f;
  unsigned kept = 0;
  if constexpr (COMBINE) {
    const int lane = threadIdx.x & 31;
    if (lane < a.k) {
      my_row = __ldg(a.row_of + t * a.k + lane);
      if (my_row >= a.rows_max) {
        record_error(a.err, MOE_DEVERR_ROW);
        my_row = -1;
      }
      if (a.topk_gate) my_gate = __ldg(a.topk_gate + t * a.k + lane);
    }
    kept = __ballot_sync(kFull, my_row >= 0);
  }
  Oct x[V], b[V];
  f32x2 ss2 = both(0.f);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = threadIdx.x + v * blockDim.x;
    x[v] = b[v] = oct_const(0.f);
    const bool in_row = c < n8;
    if (!COMBINE && !in_row) continue;
    Raw8<RT> r;
    if (in_row) r.load(a.r, t * a.d + c * 8);
    if constexpr (COMBINE) {
      // the kept slots in order, R at a time: all their loads, then the sums
      constexpr int R = 4;
      for (unsigned left = kept; left; left &= left - 1) {
        Raw8<YT> in[R];
        int slot[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
          slot[j] = -1;
          if (left) {
            slot[j] = __ffs(left) - 1;
            const long long row = __shfl_sync(kFull, my_row, slot[j]);   // by the whole warp
            if (in_row) in[j].load(a.y, row * a.d + c * 8);
            if (j + 1 < R) left &= left - 1;             // the loop drops the last one
          }
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
          if (slot[j] < 0) continue;
          // without gates the factor is one: the product is exact, the sum rounds as an addition
          const f32x2 g = both(__shfl_sync(kFull, my_gate, slot[j]));
          const Oct o = in[j].oct();
#pragma unroll
          for (int i = 0; i < 4; ++i) b[v].p[i] = fma2(g, o.p[i], b[v].p[i]);
        }
      }
      if (!in_row) {
        b[v] = oct_const(0.f);                           // sums of nothing that was loaded
        continue;
      }
      if (a.shared_y) {
        Raw8<YT> in;
        in.load(a.shared_y, t * a.d + c * 8);
        const Oct o = in.oct();
#pragma unroll
        for (int i = 0; i < 4; ++i) b[v].p[i] = add2(b[v].p[i], o.p[i]);
      }
      if (a.y_out) store_oct<YT>(a.y_out, t * a.d + c * 8, b[v]);
    } else if (a.y) {
      Raw8<YT> in;
      in.load(a.y, t * a.d + c * 8);
      b[v] = in.oct();
    }
    x[v] = r.oct();
#pragma unroll
    for (int i = 0; i < 4; ++i) ss2 = fma2(b[v].p[i], b[v].p[i], ss2);
  }
  f32x2 ry = both(1.f);
  if (a.post) ry = both(inv_rms(block_sum(sum2(ss2), part[0], warps), a.inv_d, a.eps));
  const float* gate = a.gate ? a.gate + (long long)((int)t / a.per_gate) * a.d : nullptr;
  const f32x2 alpha = both(a.alpha);
  ss2 = both(0.f);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = threadIdx.x + v * blockDim.x;
    if (c >= n8) continue;
    const Oct p = param8(a.post, c * 8), q = param8(gate, c * 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 br = mul2(mul2(mul2(b[v].p[i], ry), p.p[i]), q.p[i]);
      x[v].p[i] = fma2(alpha, x[v].p[i], br);
      ss2 = fma2(x[v].p[i], x[v].p[i], ss2);
    }
    if (a.x_out) store_oct<RT>(a.x_out, t * a.d + c * 8, x[v]);
  }
  if (a.pre) {
    const f32x2 rx = both(inv_rms(block_sum(sum2(ss2), part[1], warps), a.inv_d, a.eps));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = threadIdx.x + v * blockDim.x;
      if (c >= n8) continue;
      Oct p = param8(a.pre, c * 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) p.p[i] = mul2(mul2(x[v].p[i], rx), p.p[i]);
      store_oct<NT>(a.n_out, t * a.d + c * 8, p);
    }
  }
}

struct NormGradArgs {
  const void* d_x;            // [T, d] or null
  const void* d_n;            // [T, d] or null
  const void* x_out;          // [T, d] or null
  const void* y;              // [T, d] or null
  const float* post;
  const float* gate;
  const float* pre;
  void* d_r;                  // [T, d]
  void* d_y;                  // [T, d] or null
  float* d_gate;              // [G, d] or null
  float* p_post;              // [blocks, d] or null: the blocks' sums
  float* p_pre;               // [blocks, d] or null
  float* p_gate;              // [blocks, 2, d]: a block's part of a gate group it shares (edge_slot)
  float alpha, eps, inv_d;
  int T, d, per_gate, stages;
  int* err;
};

constexpr int kGradStages = 4;

// Tokens [row_begin(b), row_begin(b + 1)) are block b's.
__host__ __device__ __forceinline__ int row_begin(long long T, int b, int blocks) { return (int)(T * b / blocks); }

// Eight elements of a row in shared memory.
template <typename T>
__device__ __forceinline__ Oct row8(const uint8_t* base, int c) {
  if constexpr (sizeof(T) == 2) {
    return oct_bf16(*reinterpret_cast<const uint4*>(base + c * 16));
  } else {
    return oct_f32(*reinterpret_cast<const uint4*>(base + c * 32), *reinterpret_cast<const uint4*>(base + c * 32 + 16));
  }
}
// Eight parameters in shared memory, the first four and the last four of each eight in two halves
// of the buffer, so that neighbouring threads' 16 bytes are neighbours.
__device__ __forceinline__ Oct halves8(const uint8_t* base, int d, int c) {
  const uint8_t* p = base + c * 16;
  return oct_f32(*reinterpret_cast<const uint4*>(p), *reinterpret_cast<const uint4*>(p + d * 2));
}
__device__ __forceinline__ void put_halves8(uint8_t* base, int d, int c, const Oct& o) {
  const float2 a = unpack2(o.p[0]), b = unpack2(o.p[1]), e = unpack2(o.p[2]), f = unpack2(o.p[3]);
  *reinterpret_cast<float4*>(base + c * 16) = make_float4(a.x, a.y, b.x, b.y);
  *reinterpret_cast<float4*>(base + d * 2 + c * 16) = make_float4(e.x, e.y, f.x, f.y);
}
__device__ __forceinline__ void bulk_row(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// A block takes an equal run of tokens, whatever the gate groups.  Its rows arrive in a ring of
// `stages` shared-memory buffers by bulk copies issued by thread 0, so that the next rows load
// while a row is reduced; each phase reads what it needs from there, and u, h and the column sums
// stay in registers.  A buffer is filled again once every thread is past the row after it (the
// barrier of that row's first reduction), or, with one buffer, past the row itself.
// gate * post of the current gate group and pre wait in shared memory (each thread its own columns):
// the rows leave little of the first-level cache for them.  pre costs some widths a stage (with an
// fp32 residual and bf16 y and n: 8192 two to one), and gains at others (4096 x 7168: 110 -> 105 us).
template <typename YT, typename RT, typename NT, int V>
__global__ void __launch_bounds__(V == 1 ? 64 : 512, V == 1 ? 12 : 1)
block_norm_grad_kernel(const NormGradArgs a) {
  extern __shared__ __align__(16) uint8_t nsm[];
  __shared__ float2 part[2][2][kNormMaxWarps];
  __shared__ __align__(8) uint64_t s_bar[kGradStages];
  __shared__ int s_abort;
  const int warps = blockDim.x >> 5;
  const int n8 = a.d >> 3;
  const uint32_t rb = (uint32_t)a.d * sizeof(RT), nb = (uint32_t)a.d * sizeof(NT), yb = (uint32_t)a.d * sizeof(YT);
  // a stage: d_x, x_out, d_n, y, as far as they are given
  const uint32_t o_x = a.d_x ? rb : 0, o_n = o_x + (a.pre ? rb : 0), o_y = o_n + (a.pre ? nb : 0);
  const uint32_t stage_bytes = o_y + (a.y ? yb : 0);
  uint8_t* s_w = nsm + (uint32_t)a.stages * stage_bytes;   // gate * post, fp32 [d]
  uint8_t* s_p = s_w + (a.y ? (uint32_t)a.d * 4 : 0);      // pre, fp32 [d]
  const uint32_t bar0 = smem_u32(s_bar), buf0 = smem_u32(nsm);
  volatile int* abort_flag = &s_abort;
  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int s = 0; s < a.stages; ++s) mbar_init(bar0 + 8 * s, 1);
    fence_mbar_init();
  }
  __syncthreads();
  const int t0 = row_begin(a.T, blockIdx.x, gridDim.x), t1 = row_begin(a.T, blockIdx.x + 1, gridDim.x);
  int load_t = t0, load_slot = 0;                          // thread 0: the next row to load
  auto issue = [&]() {
    if (load_t >= t1 || *abort_flag) return;
    const uint32_t bar = bar0 + 8 * load_slot, dst = buf0 + (uint32_t)load_slot * stage_bytes;
    const long long at = (long long)load_t * a.d;
    mbar_expect_tx(bar, stage_bytes);
    if (a.d_x) bulk_row(dst, static_cast<const RT*>(a.d_x) + at, rb, bar);
    if (a.pre) {
      bulk_row(dst + o_x, static_cast<const RT*>(a.x_out) + at, rb, bar);
      bulk_row(dst + o_n, static_cast<const NT*>(a.d_n) + at, nb, bar);
    }
    if (a.y) bulk_row(dst + o_y, static_cast<const YT*>(a.y) + at, yb, bar);
    ++load_t;
    if (++load_slot == a.stages) load_slot = 0;
  };
  if (threadIdx.x == 0)
    for (int s = 0; s < (a.stages > 1 ? a.stages - 1 : 1); ++s) issue();

  Oct s_pre[V], s_uy[V];                                   // sum_t d_n xh; sum_t u yh over the gate group
#pragma unroll
  for (int v = 0; v < V; ++v) s_pre[v] = s_uy[v] = oct_const(0.f);
  const f32x2 alpha = both(a.alpha);
  int buf = 0, slot = 0;
  uint32_t parity = 0;
  int g = -1, g_end = t0;                                  // the current gate group, its last token + 1
  bool any_post = false;
  // the group's sums: d_gate = post * sum u yh (whole if the group is all this block's, else the
  // block's part), and gate * the same onto the block's d_post
  auto close_group = [&]() {
    const bool whole = g * a.per_gate >= t0 && g_end <= t1;
    const int edge = g * a.per_gate < t0 ? 0 : 1;          // it began before this block, or here
    float* to = !a.d_gate ? nullptr
                : whole   ? a.d_gate + (long long)g * a.d
                          : a.p_gate + ((long long)blockIdx.x * 2 + edge) * a.d;
    const float* gate = a.gate ? a.gate + (long long)g * a.d : nullptr;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = threadIdx.x + v * blockDim.x;
      if (c >= n8) continue;
      const Oct p = param8(a.post, c * 8), q = param8(gate, c * 8);
      if (a.p_post) {
        float* at = a.p_post + (long long)blockIdx.x * a.d + c * 8;
        Oct o = oct_const(0.f);
        if (any_post) o = oct_f32(*reinterpret_cast<const uint4*>(at), *reinterpret_cast<const uint4*>(at + 4));
#pragma unroll
        for (int i = 0; i < 4; ++i) o.p[i] = fma2(q.p[i], s_uy[v].p[i], o.p[i]);
        store_oct<float>(at, 0, o);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) s_uy[v].p[i] = mul2(s_uy[v].p[i], p.p[i]);
      if (to) store_oct<float>(to, c * 8, s_uy[v]);
      s_uy[v] = oct_const(0.f);
    }
    any_post = true;
  };
  if (a.pre) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = threadIdx.x + v * blockDim.x;
      if (c < n8) put_halves8(s_p, a.d, c, param8(a.pre, c * 8));
    }
  }
  for (int t = t0; t < t1; ++t, buf ^= 1) {
    if (t == g_end && a.y) {
      if (g >= 0) close_group();
      g = t / a.per_gate;
      g_end = (g + 1) * a.per_gate;
      const float* gate = a.gate ? a.gate + (long long)g * a.d : nullptr;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = threadIdx.x + v * blockDim.x;
        if (c >= n8) continue;
        const Oct p = param8(a.post, c * 8);
        Oct q = param8(gate, c * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) q.p[i] = mul2(q.p[i], p.p[i]);
        put_halves8(s_w, a.d, c, q);
      }
    }
    const long long at = (long long)t * a.d;
    const uint8_t* st = nsm + (uint32_t)slot * stage_bytes;
    Oct u[V];                                              // pre * d_n first
    if (a.pre) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = threadIdx.x + v * blockDim.x;
        u[v] = c < n8 ? halves8(s_p, a.d, c) : oct_const(0.f);
      }
    }
    mbar_wait(bar0 + 8 * slot, parity, abort_flag, a.err);
    if (++slot == a.stages) { slot = 0; parity ^= 1u; }
    f32x2 rx = both(0.f), mx = both(0.f);
    if (a.pre) {
      f32x2 xx = both(0.f), gx = both(0.f);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = threadIdx.x + v * blockDim.x;
        if (c >= n8) continue;
        const Oct x = row8<RT>(st + o_x, c), dn = row8<NT>(st + o_n, c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u[v].p[i] = mul2(u[v].p[i], dn.p[i]);
          xx = fma2(x.p[i], x.p[i], xx);
          gx = fma2(u[v].p[i], x.p[i], gx);
        }
      }
      const float2 s = block_sum2(sum2(xx), sum2(gx), part[buf][0], warps);
      const float r = inv_rms(s.x, a.inv_d, a.eps);
      rx = both(r);
      mx = both(-(s.y * r * a.inv_d * r));              // minus mean(g xh) / rms, for xh
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) u[v] = oct_const(0.f);
      __syncthreads();
    }
    if (a.stages > 1 && threadIdx.x == 0) issue();         // into the row before's buffer
    f32x2 yy = both(0.f), hy = both(0.f);
    Oct h[V];                                              // u gate post
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = threadIdx.x + v * blockDim.x;
      if (c >= n8) continue;
      if (a.pre) {
        const Oct x = row8<RT>(st + o_x, c), dn = row8<NT>(st + o_n, c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x2 xh = mul2(x.p[i], rx);
          s_pre[v].p[i] = fma2(dn.p[i], xh, s_pre[v].p[i]);
          u[v].p[i] = fma2(mx, xh, mul2(rx, u[v].p[i]));
        }
      }
      if (a.d_x) {
        const Oct dx = row8<RT>(st, c);
#pragma unroll
        for (int i = 0; i < 4; ++i) u[v].p[i] = add2(u[v].p[i], dx.p[i]);
      }
      Oct o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o.p[i] = mul2(alpha, u[v].p[i]);
      store_oct<RT>(a.d_r, at + c * 8, o);
      if (!a.y) continue;
      const Oct y = row8<YT>(st + o_y, c), w = halves8(s_w, a.d, c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[v].p[i] = mul2(u[v].p[i], w.p[i]);
        yy = fma2(y.p[i], y.p[i], yy);
        hy = fma2(h[v].p[i], y.p[i], hy);
      }
    }
    if (a.y) {
      // without a post-norm: 1 / rms = 1 and no mean
      f32x2 ry = both(1.f), my = both(0.f);
      if (a.post) {
        const float2 s = block_sum2(sum2(yy), sum2(hy), part[buf][1], warps);
        const float r = inv_rms(s.x, a.inv_d, a.eps);
        ry = both(r);
        my = both(-(s.y * r * a.inv_d * r));            // minus mean(h yh) / rms, for yh
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = threadIdx.x + v * blockDim.x;
        if (c >= n8) continue;
        const Oct y = row8<YT>(st + o_y, c);
        Oct o = h[v];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x2 yh = mul2(y.p[i], ry);
          s_uy[v].p[i] = fma2(u[v].p[i], yh, s_uy[v].p[i]);
          if (a.post) o.p[i] = fma2(my, yh, mul2(ry, h[v].p[i]));
        }
        store_oct<YT>(a.d_y, at + c * 8, o);
      }
    }
    if (a.stages == 1) {
      __syncthreads();
      if (threadIdx.x == 0) issue();
    }
  }
  if (a.y && t1 > t0) close_group();
  if (a.p_pre) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = threadIdx.x + v * blockDim.x;
      if (c < n8) store_oct<float>(a.p_pre, (long long)blockIdx.x * a.d + c * 8, s_pre[v]);
    }
  }
  // after a timeout loads may be left in flight: let them land before the block's memory is reused
  if (threadIdx.x == 0 && *abort_flag) {
    const int loaded = load_t - t0;
    for (int r = loaded > a.stages ? loaded - a.stages : 0; r < loaded; ++r)
      mbar_wait_drain(bar0 + 8 * (r % a.stages), (uint32_t)(r / a.stages) & 1u, a.err);
  }
}

// Column sums of partial rows in a fixed order: a block has 64 columns (two a lane) and 16 slices
// of the rows, each added in fp32 (at most 12 blocks a multiprocessor: 111 rows), the slices in
// fp64.  blockIdx.y 0 and 1: the post and pre weights', over all blocks' rows.  From 2 on: a gate
// group that two or more blocks share; its own part (slot 1) of the block that begins it and the
// parts (slot 0) of the blocks after.  Those groups are found among the groups, or among the
// blocks' last groups, whichever are fewer.
struct ColumnArgs {
  const float* post;          // [blocks, d], or null
  const float* pre;
  const float* gate;          // [blocks, 2, d], or null
  float* d_post;
  float* d_pre;
  float* d_gate;
  int blocks, d, T, per_gate, by_group;
};
constexpr int kSlices = 16;

// The block that token t is in: the last one that begins at or before it.
__device__ __forceinline__ int block_of(int t, int T, int blocks) {
  return (int)(((long long)(t + 1) * blocks + T - 1) / T) - 1;
}
__global__ void __launch_bounds__(32 * kSlices)
column_sum_kernel(const ColumnArgs a) {
  __shared__ float s[kSlices][66];
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");        // the sums' kernel is done, its stores visible
  const float* in;
  float* out;
  long long first = 0, step = a.d;
  int n = a.blocks;
  if (blockIdx.y < 2) {
    in = blockIdx.y ? a.pre : a.post;
    out = blockIdx.y ? a.d_pre : a.d_post;
    if (!in) return;
  } else {
    int b = blockIdx.y - 2;
    const int g = a.by_group ? b : (row_begin(a.T, b + 1, a.blocks) - 1) / a.per_gate;
    const int begin = g * a.per_gate, end = begin + a.per_gate;
    if (a.by_group) b = block_of(begin, a.T, a.blocks);
    if (begin < row_begin(a.T, b, a.blocks)) return;       // another block begins it
    const int last = block_of(end - 1, a.T, a.blocks);
    if (last == b) return;                                 // its block wrote the gradient
    n = last - b + 1;
    in = a.gate + (long long)b * 2 * a.d;
    first = a.d;                                           // slot 1 of block b, then slots 0
    step = 2LL * a.d;
    out = a.d_gate + (long long)g * a.d;
  }
  const int c = blockIdx.x * 64 + lane * 2;
  float2 acc = make_float2(0.f, 0.f);
  if (c < a.d) {
    for (int i0 = part; i0 < n; i0 += 8 * kSlices) {
      float2 f[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = i0 + kSlices * k;
        // a coherent load: these lines were written while this kernel was already resident
        f[k] = i < n ? __ldcg(reinterpret_cast<const float2*>(in + (i ? i * step : first) + c)) : make_float2(0.f, 0.f);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        acc.x += f[k].x;
        acc.y += f[k].y;
      }
    }
  }
  s[part][lane * 2] = acc.x;
  s[part][lane * 2 + 1] = acc.y;
  __syncthreads();
  const int cc = blockIdx.x * 64 + threadIdx.x;
  if (threadIdx.x < 64 && cc < a.d) {
    double sum = (double)s[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < kSlices; ++i) sum += (double)s[i][threadIdx.x];
    out[cc] = (float)sum;
  }
}

// Threads and vectors for a row of n8 <= 1024 vectors of eight: one vector a thread up to 256
// threads, two beyond.
struct Shape {
  int V, threads;
};
Shape row_shape(int n8) {
  Shape s;
  s.V = n8 <= 256 ? 1 : 2;
  s.threads = ((n8 + s.V - 1) / s.V + 31) / 32 * 32;
  return s;
}

// The backward pass: two vectors a thread from 64 on, so that a row's two reductions are shared by
// half the warps (d = 2048: 54 us against 62 with one).
Shape grad_shape(int n8) {
  Shape s;
  s.V = n8 <= 64 ? 1 : 2;
  s.threads = ((n8 + s.V - 1) / s.V + 31) / 32 * 32;
  return s;
}

template <typename YT, typename RT, typename NT, bool COMBINE>
moe_status run_norm(const NormArgs& a, cudaStream_t s) {
  const Shape sh = row_shape(a.d / 8);
  // a block for each row: they start as others end, so no wave of them is left half empty
  const long long blocks = a.T;
  if (sh.V == 1) block_norm_kernel<YT, RT, NT, 1, COMBINE><<<(unsigned)blocks, sh.threads, 0, s>>>(a);
  else block_norm_kernel<YT, RT, NT, 2, COMBINE><<<(unsigned)blocks, sh.threads, 0, s>>>(a);
  return check_launch();
}

template <typename YT, bool COMBINE>
moe_status norm_types(const NormArgs& a, int r_dtype, int n_dtype, cudaStream_t s) {
  if (r_dtype == MOE_F32)
    return n_dtype == MOE_F32 ? run_norm<YT, float, float, COMBINE>(a, s)
                              : run_norm<YT, float, __nv_bfloat16, COMBINE>(a, s);
  return n_dtype == MOE_F32 ? run_norm<YT, __nv_bfloat16, float, COMBINE>(a, s)
                            : run_norm<YT, __nv_bfloat16, __nv_bfloat16, COMBINE>(a, s);
}

// Blocks of the backward pass: what the device holds at once (a multiprocessor: 512 threads of
// two vectors each, or up to 12 small blocks of one), at most one a token.
struct GradPlan {
  int blocks, per_sm;
};
GradPlan grad_plan(int T, int d) {
  GradPlan p;
  const Shape sh = grad_shape(d / 8);
  p.per_sm = (sh.V == 1 ? 768 : 512) / sh.threads;         // at least 1
  if (p.per_sm > 12) p.per_sm = 12;
  const int want = p.per_sm * num_sms();
  p.blocks = T < want ? T : want;
  return p;
}

template <typename YT, typename RT, typename NT, int V>
moe_status run_grad_v(NormGradArgs a, const GradPlan& p, int threads, cudaStream_t s) {
  constexpr size_t kSmem = 226 * 1024;                     // a multiprocessor's, less the static part
  static std::atomic<int> configured[kMaxDevices];
  const moe_status st = ensure_smem_limit(configured, block_norm_grad_kernel<YT, RT, NT, V>, kSmem);
  if (st != MOE_OK) return st;
  const size_t row = (size_t)a.d * ((a.d_x ? sizeof(RT) : 0) + (a.pre ? sizeof(RT) + sizeof(NT) : 0) +
                                    (a.y ? sizeof(YT) : 0));   // at most 128 KB: one always fits
  const size_t w = (size_t)a.d * sizeof(float) * ((a.y ? 1 : 0) + (a.pre ? 1 : 0));
  const size_t room = kSmem / p.per_sm - 2048 - w;
  a.stages = (int)(room / row);
  if (a.stages > kGradStages) a.stages = kGradStages;
  if (a.stages < 1) a.stages = 1;
  block_norm_grad_kernel<YT, RT, NT, V><<<p.blocks, threads, a.stages * row + w, s>>>(a);
  return check_launch();
}

template <typename YT, typename RT, typename NT>
moe_status run_grad(const NormGradArgs& a, const GradPlan& p, cudaStream_t s) {
  const Shape sh = grad_shape(a.d / 8);
  if (sh.V == 1) return run_grad_v<YT, RT, NT, 1>(a, p, sh.threads, s);
  return run_grad_v<YT, RT, NT, 2>(a, p, sh.threads, s);
}

}  // namespace

moe_status launch_block_norm(const void* r, int r_dtype, const void* y, int y_dtype, const int32_t* row_of,
                             const float* topk_gate, const void* shared_y, int k, long long rows_max, void* y_out,
                             const float* post, const float* gate, int G, float alpha, const float* pre, float eps,
                             int T, int d, void* x_out, void* n_out, int n_dtype, cudaStream_t s) {
  NormArgs a{r, y, post, gate, pre, row_of, topk_gate, shared_y, y_out, x_out, n_out, rows_max, alpha, eps,
             1.f / (float)d, T, d, gate ? T / G : 1, k, err_ptr()};
  if (row_of)
    return y_dtype == MOE_F32 ? norm_types<float, true>(a, r_dtype, n_dtype, s)
                              : norm_types<__nv_bfloat16, true>(a, r_dtype, n_dtype, s);
  return y_dtype == MOE_F32 ? norm_types<float, false>(a, r_dtype, n_dtype, s)
                            : norm_types<__nv_bfloat16, false>(a, r_dtype, n_dtype, s);
}

// Each block's sums: the post and pre weights', and its parts of at most two gate groups that it
// shares with its neighbours.
size_t block_norm_grad_workspace_bytes(int T, int d) {
  return (size_t)4 * grad_plan(T, d).blocks * d * sizeof(float);
}

moe_status launch_block_norm_backward(const void* d_x, const void* d_n, const void* x_out, const void* y, int y_dtype,
                                      int r_dtype, int n_dtype, const float* post, const float* gate, int G,
                                      float alpha, const float* pre, float eps, int T, int d, void* d_r, void* d_y,
                                      float* d_post, float* d_gate, float* d_pre, void* ws, cudaStream_t s) {
  const GradPlan p = grad_plan(T, d);
  float* w = static_cast<float*>(ws);
  const size_t one = (size_t)p.blocks * d;
  NormGradArgs a{d_x, d_n, x_out, y, post, gate, pre, d_r, d_y, d_gate, d_post ? w : nullptr, d_pre ? w + one : nullptr,
                 w + 2 * one, alpha, eps, 1.f / (float)d, T, d, T / G, 1, err_ptr()};
  moe_status st;
  if (y_dtype == MOE_F32) {
    if (r_dtype == MOE_F32)
      st = n_dtype == MOE_F32 ? run_grad<float, float, float>(a, p, s)
                              : run_grad<float, float, __nv_bfloat16>(a, p, s);
    else
      st = n_dtype == MOE_F32 ? run_grad<float, __nv_bfloat16, float>(a, p, s)
                              : run_grad<float, __nv_bfloat16, __nv_bfloat16>(a, p, s);
  } else {
    if (r_dtype == MOE_F32)
      st = n_dtype == MOE_F32 ? run_grad<__nv_bfloat16, float, float>(a, p, s)
                              : run_grad<__nv_bfloat16, float, __nv_bfloat16>(a, p, s);
    else
      st = n_dtype == MOE_F32 ? run_grad<__nv_bfloat16, __nv_bfloat16, float>(a, p, s)
                              : run_grad<__nv_bfloat16, __nv_bfloat16, __nv_bfloat16>(a, p, s);
  }
  if (st != MOE_OK) return st;
  if (!d_post && !d_gate && !d_pre) return MOE_OK;
  const bool shared = d_gate && G < T;                     // a group of one token is never shared
  const bool by_group = G <= p.blocks;
  const ColumnArgs c{a.p_post, a.p_pre, a.p_gate, d_post, d_pre, d_gate, p.blocks, d, T, T / G, by_group};
  // its launch overlaps the end of the kernel before it (53.5 -> 50.4 us at 8192 x 2048)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((d + 63) / 64, 2 + (shared ? by_group ? G : p.blocks : 0));
  cfg.blockDim = dim3(32 * kSlices);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, column_sum_kernel, c));
}

}  // namespace moe
