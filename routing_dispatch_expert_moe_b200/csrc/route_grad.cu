// Gradient of a routing by its logits: the gates', the load-balancing loss's and the router
// z-loss's.
//
// "Hugging Face 图解 Mixture of Experts（MoE）原理、训练与推理权衡", section "什么是稀疏性？"
// (gates), the sections on the load-balancing loss, and "使用路由器 Z-loss 稳定训练"; handbook
// news post (hub.geekagi.cn), quoted tweet (softmax, sigmoid, sqrt(softplus)).
//
// For one token with logits l, selected experts i_j, upstream gate gradients u_j (scale folded
// in), scores s_e = s(l_e), p = softmax(l):
//   softmax, renormalised     q = softmax over the selected;  dl_{i_j} += q_j (u_j - sum_i q_i u_i)
//   softmax                   dl_e += [e = i_j] p_e u_j - p_e sum_j p_{i_j} u_j
//   others, renormalised      S = sum_j s_{i_j};  dl_{i_j} += s'_{i_j} (u_j - sum_i s_i u_i / S) / S
//   others                    dl_{i_j} += s'_{i_j} u_j
//   load balance              c = aux E / T;  dl_e += c p_e (f_e - sum f p)            (softmax)
//                             dl_e += c s'_e (f_e - sum f s / sum s) / sum s           (others)
//   z-loss                    dl_e += 2 z / T lse p_e
// A masked logit (-inf or NaN) has gradient zero, a row of them only zeros.
//
// It reads each logit once and writes each gradient once: 8E bytes a token, bound by HBM with
// the exponentials close behind.  One warp per token keeps the row in registers; the selected
// experts' terms meet the dense ones through a row of shared memory.
#include <float.h>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kGradWarps = 8;
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float wmax(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
__device__ __forceinline__ float wsum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ float clean_logit(float l) { return l > -INFINITY ? fminf(l, FLT_MAX) : -INFINITY; }

// Score and derivative of the two scores that act on one logit alone; both 0 at -inf.  With
// e = exp(-|l|): sigmoid = 1 / (1 + e) or e / (1 + e), and its derivative e / (1 + e)^2.
__device__ __forceinline__ void score_grad(float l, int score, float* s, float* ds) {
  const float e = expf(-fabsf(l));
  const float r = 1.f / (1.f + e);
  const float sig = l >= 0.f ? r : e * r;
  if (score == MOE_SCORE_SIGMOID) {
    *s = sig;
    *ds = e * r * r;
  } else {
    const float root = sqrtf(fmaxf(l, 0.f) + log1pf(e));
    *s = root;
    *ds = root > 0.f ? sig / (2.f * root) : 0.f;
  }
}

struct GradArgs {
  const float* logits;
  const int32_t* topk_idx;
  const float* d_gate;
  const float* load;
  float* d_logits;
  int T, E, k, score, renorm;
  float scale, aux, z;     // aux = aux_coef * E / T, z = 2 * z_coef / T
  int* err;
};

// NV: vectors of four logits a lane holds (VEC), or single ones.
template <int NV, bool VEC>
__global__ void __launch_bounds__(32 * kGradWarps)
route_grad_kernel(const GradArgs a) {
  constexpr int W = VEC ? 4 : 1;
  constexpr int N = NV * W;
  extern __shared__ __align__(16) float rsm[];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int E = a.E, k = a.k;
  float* add = rsm + (size_t)w * ((E + 3) / 4 * 4);       // the selected experts' terms; zero in between
  for (int e = lane; e < E; e += 32) add[e] = 0.f;
  __syncwarp();
  auto at = [&](int i) { return VEC ? 4 * (lane + 32 * (i / 4)) + i % 4 : lane + 32 * i; };
  const bool sm = a.score == MOE_SCORE_SOFTMAX;
  const bool gates = a.d_gate != nullptr;
  const bool aux = a.aux != 0.f, zl = a.z != 0.f;
  const bool need_p = (sm && (aux || (gates && !a.renorm))) || zl;   // the full softmax
  const bool need_s = !sm && aux;                                    // every expert's score
  const long long nw = (long long)gridDim.x * kGradWarps;
  for (long long t = (long long)blockIdx.x * kGradWarps + w; t < a.T; t += nw) {
    const float* l = a.logits + t * E;
    float v[N];
#pragma unroll
    for (int i = 0; i < N; i += W) {
      const int e = at(i);
      if constexpr (VEC) {
        const float4 q = e < E ? __ldg(reinterpret_cast<const float4*>(l + e))
                               : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        v[i] = clean_logit(q.x); v[i + 1] = clean_logit(q.y);
        v[i + 2] = clean_logit(q.z); v[i + 3] = clean_logit(q.w);
      } else {
        v[i] = e < E ? clean_logit(__ldg(l + e)) : -INFINITY;
      }
    }
    // -------------------------------------------------- the selected experts, a lane each
    float p_dot = 0.f;                                     // softmax: sum_j p_{i_j} u_j
    int sel = -1;
    float lf = -INFINITY, u = 0.f;
    if (gates && lane < k) {
      sel = __ldg(a.topk_idx + t * k + lane);
      if ((unsigned)sel >= (unsigned)E) {
        record_error(a.err, MOE_DEVERR_EXPERT_ID);
        sel = -1;
      } else {
        lf = clean_logit(__ldg(l + sel));
        u = a.scale * __ldg(a.d_gate + t * k + lane);
      }
    }
    float m = -INFINITY, lse = 0.f, iz = 0.f;
    if (need_p) {
#pragma unroll
      for (int i = 0; i < N; ++i) m = fmaxf(m, v[i]);
      m = wmax(m);
      if (m > -INFINITY) {
        float zs = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) zs += expf(v[i] - m);
        zs = wsum(zs);
        iz = 1.f / zs;
        lse = m + logf(zs);
      }
    }
    const bool live = m > -INFINITY;
    if (gates) {
      float dk = 0.f;
      if (sm && a.renorm) {
        const float mk = wmax(lf);
        const float ex = lf > -INFINITY ? expf(lf - mk) : 0.f;
        const float tot = wsum(ex);
        const float q = tot > 0.f ? ex / tot : 0.f;
        dk = q * (u - wsum(q * u));
      } else if (sm) {
        dk = lf > -INFINITY ? expf(lf - m) * iz * u : 0.f;
        p_dot = wsum(dk);
      } else {
        float s = 0.f, ds = 0.f;
        if (lf > -INFINITY) score_grad(lf, a.score, &s, &ds);
        if (a.renorm) {
          const float tot = wsum(s), dot = wsum(s * u);
          dk = tot > 0.f ? ds * (u - dot / tot) / tot : 0.f;
        } else {
          dk = ds * u;
        }
      }
      if (sel >= 0 && dk != 0.f) atomicAdd(add + sel, dk);   // a repeated expert's terms add up
      __syncwarp();
    }
    // -------------------------------------------------- the dense terms
    float fp = 0.f, tot = 0.f;
    if (aux) {
#pragma unroll
      for (int i = 0; i < N; i += W) {
        const int e = at(i);
        float f[W];
        if constexpr (VEC) {
          const float4 q = e < E ? __ldg(reinterpret_cast<const float4*>(a.load + e)) : make_float4(0, 0, 0, 0);
          f[0] = q.x; f[1] = q.y; f[2] = q.z; f[3] = q.w;
        } else {
          f[0] = e < E ? __ldg(a.load + e) : 0.f;
        }
#pragma unroll
        for (int c = 0; c < W; ++c) {
          if (!(v[i + c] > -INFINITY)) continue;
          float s, ds;
          if (sm) s = expf(v[i + c] - m) * iz;
          else score_grad(v[i + c], a.score, &s, &ds);
          fp = fmaf(f[c], s, fp);
          tot += s;
        }
      }
      fp = wsum(fp);
      if (need_s) {
        tot = wsum(tot);
        fp = tot > 0.f ? fp / tot : 0.f;
      }
    }
    const float it = need_s && tot > 0.f ? a.aux / tot : 0.f;
    const float zc = a.z * lse;
    float* out = a.d_logits + t * E;
#pragma unroll
    for (int i = 0; i < N; i += W) {
      const int e = at(i);
      if (e >= E) continue;
      float o[W], f[W];
      if constexpr (VEC) {
        const float4 q = *reinterpret_cast<const float4*>(add + e);
        o[0] = q.x; o[1] = q.y; o[2] = q.z; o[3] = q.w;
        if (gates) *reinterpret_cast<float4*>(add + e) = make_float4(0, 0, 0, 0);
        const float4 r = aux ? __ldg(reinterpret_cast<const float4*>(a.load + e)) : make_float4(0, 0, 0, 0);
        f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w;
      } else {
        o[0] = add[e];
        if (gates) add[e] = 0.f;
        f[0] = aux ? __ldg(a.load + e) : 0.f;
      }
#pragma unroll
      for (int c = 0; c < W; ++c) {
        const float x = v[i + c];
        if (!(x > -INFINITY)) { o[c] = 0.f; continue; }
        if (need_p && live) {
          const float p = expf(x - m) * iz;
          float dense = zc - p_dot;
          if (sm && aux) dense += a.aux * (f[c] - fp);
          o[c] = fmaf(p, dense, o[c]);
        }
        if (need_s) {
          float s, ds;
          score_grad(x, a.score, &s, &ds);
          o[c] = fmaf(it * ds, f[c] - fp, o[c]);
        }
      }
      if constexpr (VEC)
        *reinterpret_cast<float4*>(out + e) = make_float4(o[0], o[1], o[2], o[3]);
      else
        out[e] = o[0];
    }
    __syncwarp();
  }
}

template <int NV, bool VEC>
moe_status run_grad(const GradArgs& a, cudaStream_t s) {
  const size_t smem = (size_t)kGradWarps * ((a.E + 3) / 4 * 4) * sizeof(float);   // at most 32 KB
  long long blocks = ((long long)a.T + kGradWarps - 1) / kGradWarps;
  const long long cap = (long long)num_sms() * 8;
  if (blocks > cap) blocks = cap;
  route_grad_kernel<NV, VEC><<<(unsigned)blocks, 32 * kGradWarps, smem, s>>>(a);
  return check_launch();
}

}  // namespace

moe_status launch_route_backward(const float* logits, const int32_t* topk_idx, const float* d_gate, int T, int E,
                                 int k, int score, int renorm, float scale, const float* load, float aux_coef,
                                 float z_coef, float* d_logits, cudaStream_t s) {
  GradArgs a{logits, topk_idx, d_gate, load, d_logits, T, E, k, score, renorm, scale,
             (float)((double)aux_coef * E / T), (float)(2.0 * (double)z_coef / T), err_ptr()};
  const bool vec = E % 4 == 0 && aligned16(logits) && aligned16(d_logits) && aligned16(load);
  if (vec) {
    const int nv = (E / 4 + 31) / 32;                      // at most 8
    if (nv <= 1) return run_grad<1, true>(a, s);
    if (nv <= 2) return run_grad<2, true>(a, s);
    if (nv <= 4) return run_grad<4, true>(a, s);
    if (nv <= 7) return run_grad<7, true>(a, s);
    return run_grad<8, true>(a, s);
  }
  const int nv = (E + 31) / 32;                            // at most 32
  if (nv <= 2) return run_grad<2, false>(a, s);
  if (nv <= 8) return run_grad<8, false>(a, s);
  return run_grad<32, false>(a, s);
}

}  // namespace moe
