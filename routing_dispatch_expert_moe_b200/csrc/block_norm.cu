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
// registers.  A block of TPR threads has a row; a thread has V vectors of eight neighbouring
// elements.  Sums are fp32: a thread's elements, a shuffle, then the warps' sums through shared
// memory.  The backward pass gives each block a run of rows of one gate group; it keeps the
// weights' column sums in registers over all its rows and writes them out once, and a second
// kernel adds the blocks' partial sums in a fixed order in fp64 (results repeat bit for bit).
#include "common.cuh"
#include "row8.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kNormMaxWarps = 16;

// Sum of two values over the block; `part` is this call's own slice of shared
// memory, so that a row needs one barrier for each reduction.
__device__ __forceinline__ float2 block_sum2(float a, float b, float2* part, int warps) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(kFull, a, o);
    b += __shfl_xor_sync(kFull, b, o);
  }
  if (warps == 1) return make_float2(a, b);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  if (lane == 0) part[w] = make_float2(a, b);
  __syncthreads();
  float2 s = lane < warps ? part[lane] : make_float2(0.f, 0.f);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    s.x += __shfl_xor_sync(kFull, s.x, o);
    s.y += __shfl_xor_sync(kFull, s.y, o);
  }
  return s;
}

template <typename T>
__device__ __forceinline__ void load8(const void* base, long long e, float* f) {
  Row8<T> r;
  r.load(base, e);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = 0.f;
  r.add(f, 1.f, false);
}
__device__ __forceinline__ void param8(const float* p, long long e, float* f) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p + e));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p + e + 4));
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
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
  float alpha, eps;
  int T, d, per_gate, k;      // per_gate: tokens that share a gate row
  int* err;
};

// YT: y or the expert rows; RT: the residual stream; NT: the normed rows.
template <typename YT, typename RT, typename NT, int V, bool COMBINE>
__global__ void __launch_bounds__(V == 1 ? 256 : 512)
block_norm_kernel(const NormArgs a) {
  __shared__ float2 part[2][2][kNormMaxWarps];
  __shared__ int s_row[2][32];
  __shared__ float s_w[2][32];
  const int warps = blockDim.x >> 5;
  const int n8 = a.d >> 3;
  int buf = 0;
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x, buf ^= 1) {
    int nk = 0;
    if constexpr (COMBINE) {
      // the token's kept rows, in slot order
      if (threadIdx.x < 32) {
        int row = -1;
        float g = 1.f;
        if (threadIdx.x < a.k) {
          row = __ldg(a.row_of + t * a.k + threadIdx.x);
          if (row >= a.rows_max) { record_error(a.err, MOE_DEVERR_ROW); row = -1; }
          if (a.topk_gate) g = __ldg(a.topk_gate + t * a.k + threadIdx.x);
        }
        const unsigned kept = __ballot_sync(kFull, row >= 0);
        s_row[buf][threadIdx.x] = -1;
        __syncwarp();
        if (row >= 0) {
          const int at = __popc(kept & ((1u << threadIdx.x) - 1u));
          s_row[buf][at] = row;
          s_w[buf][at] = g;
        }
      }
      __syncthreads();
      while (nk < a.k && s_row[buf][nk] >= 0) ++nk;
    }
    float x[V][8], b[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = threadIdx.x + v * blockDim.x;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[v][i] = b[v][i] = 0.f;
      if (c >= n8) continue;
      load8<RT>(a.r, t * a.d + c * 8, x[v]);
      if constexpr (COMBINE) {
        for (int j0 = 0; j0 < nk; j0 += 4) {               // four rows in flight
          Row8<YT> in[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j0 + j < nk) in[j].load(a.y, (long long)s_row[buf][j0 + j] * a.d + c * 8);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j0 + j < nk) in[j].add(b[v], s_w[buf][j0 + j], a.topk_gate != nullptr);
        }
        if (a.shared_y) {
          Row8<YT> in;
          in.load(a.shared_y, t * a.d + c * 8);
          in.add(b[v], 1.f, false);
        }
        if (a.y_out) store8<YT>(a.y_out, t * a.d + c * 8, b[v]);
      } else {
        if (a.y) load8<YT>(a.y, t * a.d + c * 8, b[v]);
      }
    }
    float ry = 1.f;
    if (a.post) {
      float ss = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(b[v][i], b[v][i], ss);
      ss = block_sum2(ss, 0.f, part[buf][0], warps).x;
      ry = 1.f / sqrtf(ss / (float)a.d + a.eps);
    }
    const float* gate = a.gate ? a.gate + t / a.per_gate * a.d : nullptr;
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = threadIdx.x + v * blockDim.x;
      if (c >= n8) continue;
      float p[8];
      if (a.post) {
        param8(a.post, c * 8, p);
#pragma unroll
        for (int i = 0; i < 8; ++i) b[v][i] = b[v][i] * ry * p[i];
      }
      if (gate) {
        param8(gate, c * 8, p);
#pragma unroll
        for (int i = 0; i < 8; ++i) b[v][i] *= p[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[v][i] = fmaf(a.alpha, x[v][i], b[v][i]);
        ss = fmaf(x[v][i], x[v][i], ss);
      }
      if (a.x_out) store8<RT>(a.x_out, t * a.d + c * 8, x[v]);
    }
    if (a.pre) {
      ss = block_sum2(ss, 0.f, part[buf][1], warps).x;
      const float rx = 1.f / sqrtf(ss / (float)a.d + a.eps);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = threadIdx.x + v * blockDim.x;
        if (c >= n8) continue;
        float p[8];
        param8(a.pre, c * 8, p);
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = x[v][i] * rx * p[i];
        store8<NT>(a.n_out, t * a.d + c * 8, p);
      }
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
  float* p_post;              // [blocks, d] or null
  float* p_pre;               // [blocks, d] or null
  float* p_gate;              // [G, splits, d] or null
  float alpha, eps;
  int T, d, per_gate, splits, groups;
};

template <typename YT, typename RT, typename NT, int V>
__global__ void __launch_bounds__(V == 1 ? 256 : 512)
block_norm_grad_kernel(const NormGradArgs a) {
  __shared__ float2 part[2][2][kNormMaxWarps];
  const int warps = blockDim.x >> 5;
  const int n8 = a.d >> 3;
  float s_post[V][8], s_pre[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) s_post[v][i] = s_pre[v][i] = 0.f;
  int buf = 0;
  // work item: split `sp` of gate group `g`, tokens [t0, t1)
  for (long long item = blockIdx.x; item < (long long)a.groups * a.splits; item += gridDim.x) {
    const int g = (int)(item / a.splits), sp = (int)(item - (long long)g * a.splits);
    const int t0 = g * a.per_gate + (int)((long long)a.per_gate * sp / a.splits);
    const int t1 = g * a.per_gate + (int)((long long)a.per_gate * (sp + 1) / a.splits);
    float s_gate[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) s_gate[v][i] = 0.f;
    for (int t = t0; t < t1; ++t, buf ^= 1) {
      const long long at = (long long)t * a.d;
      float u[V][8], y[V][8], x[V][8], dn[V][8];
      float xx = 0.f, gx = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = threadIdx.x + v * blockDim.x;
#pragma unroll
        for (int i = 0; i < 8; ++i) u[v][i] = y[v][i] = x[v][i] = dn[v][i] = 0.f;
        if (c >= n8) continue;
        if (a.d_x) load8<RT>(a.d_x, at + c * 8, u[v]);
        if (a.y) load8<YT>(a.y, at + c * 8, y[v]);
        if (a.pre) {
          load8<RT>(a.x_out, at + c * 8, x[v]);
          load8<NT>(a.d_n, at + c * 8, dn[v]);
          float p[8];
          param8(a.pre, c * 8, p);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            xx = fmaf(x[v][i], x[v][i], xx);
            gx = fmaf(p[i] * dn[v][i], x[v][i], gx);
          }
        }
      }
      if (a.pre) {
        const float2 s = block_sum2(xx, gx, part[buf][0], warps);
        const float rx = 1.f / sqrtf(s.x / (float)a.d + a.eps);
        const float mx = s.y * rx / (float)a.d * rx;       // mean(g xh) / rms, for x
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int c = threadIdx.x + v * blockDim.x;
          if (c >= n8) continue;
          float p[8];
          param8(a.pre, c * 8, p);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float xh = x[v][i] * rx;
            s_pre[v][i] = fmaf(dn[v][i], xh, s_pre[v][i]);
            u[v][i] += rx * (p[i] * dn[v][i]) - mx * xh;
          }
        }
      }
      const float* gate = a.gate ? a.gate + (long long)g * a.d : nullptr;
      float yy = 0.f, hy = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = threadIdx.x + v * blockDim.x;
        if (c >= n8) continue;
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = a.alpha * u[v][i];
        store8<RT>(a.d_r, at + c * 8, o);
        if (!a.y) continue;
        float p[8], q[8];
        if (a.post) param8(a.post, c * 8, p);
        if (gate) param8(gate, c * 8, q);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float h = u[v][i] * (gate ? q[i] : 1.f) * (a.post ? p[i] : 1.f);
          yy = fmaf(y[v][i], y[v][i], yy);
          hy = fmaf(h, y[v][i], hy);
        }
      }
      if (!a.y) continue;
      float ry = 1.f, my = 0.f;
      if (a.post) {
        const float2 s = block_sum2(yy, hy, part[buf][1], warps);
        ry = 1.f / sqrtf(s.x / (float)a.d + a.eps);
        my = s.y * ry / (float)a.d * ry;                   // mean(h yh) / rms, for yh
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = threadIdx.x + v * blockDim.x;
        if (c >= n8) continue;
        float p[8], q[8], o[8];
        if (a.post) param8(a.post, c * 8, p);
        if (gate) param8(gate, c * 8, q);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float yh = y[v][i] * ry;
          const float ug = u[v][i] * (gate ? q[i] : 1.f);
          s_gate[v][i] = fmaf(u[v][i], a.post ? yh * p[i] : yh, s_gate[v][i]);
          s_post[v][i] = fmaf(ug, yh, s_post[v][i]);
          o[i] = a.post ? ry * (ug * p[i]) - my * yh : ug;
        }
        store8<YT>(a.d_y, at + c * 8, o);
      }
    }
    if (a.p_gate) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = threadIdx.x + v * blockDim.x;
        if (c < n8) store8<float>(a.p_gate, item * a.d + c * 8, s_gate[v]);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = threadIdx.x + v * blockDim.x;
    if (c >= n8) continue;
    if (a.p_post) store8<float>(a.p_post, (long long)blockIdx.x * a.d + c * 8, s_post[v]);
    if (a.p_pre) store8<float>(a.p_pre, (long long)blockIdx.x * a.d + c * 8, s_pre[v]);
  }
}

// out[r, c] = sum over the n partial rows of r, in order, in fp64.  32 columns x 8 slices of
// the partial rows a block.
struct ReduceJob {
  const float* in;            // [rows, n, d]
  float* out;                 // [rows, d]
  int rows, n;
};
__global__ void __launch_bounds__(256)
column_sum_kernel(const ReduceJob j0, const ReduceJob j1, const ReduceJob j2, int d) {
  __shared__ double s[8][32];
  int r = blockIdx.y;
  ReduceJob j = j0;
  if (r >= j.rows) { r -= j.rows; j = j1; }
  if (r >= j.rows) { r -= j.rows; j = j2; }
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
  double acc = 0.0;
  if (c < d) {
    const float* p = j.in + (long long)r * j.n * d + c;
    for (int i = part; i < j.n; i += 8) acc += (double)__ldg(p + (long long)i * d);
  }
  s[part][threadIdx.x & 31] = acc;
  __syncthreads();
  if (part == 0 && c < d) {
#pragma unroll
    for (int i = 1; i < 8; ++i) acc += s[i][threadIdx.x & 31];
    j.out[(long long)r * d + c] = (float)acc;
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

template <typename YT, typename RT, typename NT, bool COMBINE>
moe_status run_norm(const NormArgs& a, cudaStream_t s) {
  const Shape sh = row_shape(a.d / 8);
  long long blocks = a.T;
  const long long cap = (long long)num_sms() * 16;
  if (blocks > cap) blocks = cap;
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

// Blocks of the backward pass and splits of a gate group: enough work items for two blocks a
// multiprocessor, never more splits than tokens.
struct GradPlan {
  int splits, blocks;
};
GradPlan grad_plan(int T, int G) {
  GradPlan p;
  const int per = T / G;
  const int want = 2 * num_sms();
  p.splits = (want + G - 1) / G;
  if (p.splits > per) p.splits = per;
  const long long items = (long long)G * p.splits;
  p.blocks = (int)(items < want ? items : want);
  return p;
}

template <typename YT, typename RT, typename NT>
moe_status run_grad(const NormGradArgs& a, int blocks, cudaStream_t s) {
  const Shape sh = row_shape(a.d / 8);
  if (sh.V == 1) block_norm_grad_kernel<YT, RT, NT, 1><<<blocks, sh.threads, 0, s>>>(a);
  else block_norm_grad_kernel<YT, RT, NT, 2><<<blocks, sh.threads, 0, s>>>(a);
  return check_launch();
}

}  // namespace

moe_status launch_block_norm(const void* r, int r_dtype, const void* y, int y_dtype, const int32_t* row_of,
                             const float* topk_gate, const void* shared_y, int k, long long rows_max, void* y_out,
                             const float* post, const float* gate, int G, float alpha, const float* pre, float eps,
                             int T, int d, void* x_out, void* n_out, int n_dtype, cudaStream_t s) {
  NormArgs a{r, y, post, gate, pre, row_of, topk_gate, shared_y, y_out, x_out, n_out, rows_max, alpha, eps, T, d,
             gate ? T / G : 1, k, err_ptr()};
  if (row_of)
    return y_dtype == MOE_F32 ? norm_types<float, true>(a, r_dtype, n_dtype, s)
                              : norm_types<__nv_bfloat16, true>(a, r_dtype, n_dtype, s);
  return y_dtype == MOE_F32 ? norm_types<float, false>(a, r_dtype, n_dtype, s)
                            : norm_types<__nv_bfloat16, false>(a, r_dtype, n_dtype, s);
}

// Partial sums: the post and pre weights' by block, the gates' by work item (a gate group that
// is one work item writes its gradient itself).
size_t block_norm_grad_workspace_bytes(int T, int d, int G) {
  const GradPlan p = grad_plan(T, G);
  return ((size_t)2 * p.blocks + (p.splits > 1 ? (size_t)G * p.splits : 0)) * d * sizeof(float);
}

moe_status launch_block_norm_backward(const void* d_x, const void* d_n, const void* x_out, const void* y, int y_dtype,
                                      int r_dtype, int n_dtype, const float* post, const float* gate, int G,
                                      float alpha, const float* pre, float eps, int T, int d, void* d_r, void* d_y,
                                      float* d_post, float* d_gate, float* d_pre, void* ws, cudaStream_t s) {
  const GradPlan p = grad_plan(T, G);
  float* w = static_cast<float*>(ws);
  NormGradArgs a{d_x, d_n, x_out, y, post, gate, pre, d_r, d_y, d_post ? w : nullptr,
                 d_pre ? w + (size_t)p.blocks * d : nullptr,
                 d_gate && p.splits > 1 ? w + (size_t)2 * p.blocks * d : d_gate,
                 alpha, eps, T, d, T / G, p.splits, G};
  moe_status st;
  if (y_dtype == MOE_F32) {
    if (r_dtype == MOE_F32)
      st = n_dtype == MOE_F32 ? run_grad<float, float, float>(a, p.blocks, s)
                              : run_grad<float, float, __nv_bfloat16>(a, p.blocks, s);
    else
      st = n_dtype == MOE_F32 ? run_grad<float, __nv_bfloat16, float>(a, p.blocks, s)
                              : run_grad<float, __nv_bfloat16, __nv_bfloat16>(a, p.blocks, s);
  } else {
    if (r_dtype == MOE_F32)
      st = n_dtype == MOE_F32 ? run_grad<__nv_bfloat16, float, float>(a, p.blocks, s)
                              : run_grad<__nv_bfloat16, float, __nv_bfloat16>(a, p.blocks, s);
    else
      st = n_dtype == MOE_F32 ? run_grad<__nv_bfloat16, __nv_bfloat16, float>(a, p.blocks, s)
                              : run_grad<__nv_bfloat16, __nv_bfloat16, __nv_bfloat16>(a, p.blocks, s);
  }
  if (st != MOE_OK) return st;
  ReduceJob jobs[3] = {{a.p_post, d_post, d_post ? 1 : 0, p.blocks},
                       {a.p_pre, d_pre, d_pre ? 1 : 0, p.blocks},
                       {a.p_gate, d_gate, d_gate && p.splits > 1 ? G : 0, p.splits}};
  const int rows = jobs[0].rows + jobs[1].rows + jobs[2].rows;
  if (rows == 0) return MOE_OK;
  column_sum_kernel<<<dim3((d + 31) / 32, rows), 256, 0, s>>>(jobs[0], jobs[1], jobs[2], d);
  return check_launch();
}

}  // namespace moe
