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
// the exponentials close behind.  One warp per token keeps the row, and of what it has computed
// once (exponentials, scores) what the second pass needs, in registers.  Rows come and go through
// two shared-memory buffers a warp by bulk copies, the next one on its way while one is worked
// on; the selected experts' terms are added to the finished row there.  32768 tokens, 896 experts,
// sigmoid with the load-balancing loss: 52 us where the bytes need 36 (151 with plain loads and
// stores); the exponentials and divisions take half of the issue rate.  8192 tokens, 64 experts:
// 7.5 us, a token's chain of reductions.  Runs of tokens a block, its warps taking the next one
// each as they come, were slower (64 against 60): neighbouring rows are better read at the same
// time.
#include <float.h>

#include "f32x2.cuh"
#include "warp_rows.cuh"

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
// NaN counts as masked (-inf; fmaxf drops a NaN), +inf as the largest float.
__device__ __forceinline__ float clean_logit(float l) { return fminf(fmaxf(l, -INFINITY), FLT_MAX); }

// exp(x) for two x <= 0 within about 3 steps: 2^(x log2 e) by the exponential unit, the rounding of
// the product and the rest of log2 e made up for to first order.  0 for -inf and below 2^-126.
__device__ __forceinline__ f32x2 exp_neg2(float x, float y) {
  constexpr float kL = 1.44269502f, kLlo = 1.92596299e-8f, kLn2 = 0.693147182f;
  const f32x2 v = pack2(fmaxf(x, -200.f), fmaxf(y, -200.f));
  const f32x2 t = mul2(v, both(kL));
  const f32x2 lo = fma2(v, both(kLlo), fma2(v, both(kL), mul2(t, both(-1.f))));
  const float2 u = unpack2(t);
  float2 r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(u.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(u.y));
  const f32x2 e = pack2(r.x, r.y);
  return fma2(e, mul2(lo, both(kLn2)), e);
}
__device__ __forceinline__ float rcp_fast(float x) {       // x in [1, 2] or a normal number: 1 step
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Score and derivative of the two scores that act on one logit alone, for two logits; 0 at -inf.
// sigmoid = r or e r with e = exp(-|l|), r = 1 / (1 + e), its derivative e r^2.
// sqrt(softplus) is sqrt(x) for l >= 0 and exp(l / 2) sqrt(x) below, x = l + log(1 + e) or
// log(1 + e) / e: the factor is a number of fp32 where e itself underflows (l < -87), down to
// l = -174.  Its derivative sigmoid / (2 sqrt(softplus)) is r / (2 sqrt(x)), times the same factor.
template <int SCORE>
__device__ __forceinline__ void score_grad2(float x, float y, f32x2* s, f32x2* ds) {
  if (SCORE == MOE_SCORE_SIGMOID) {
    const f32x2 e = exp_neg2(-fabsf(x), -fabsf(y));
    const float2 q = unpack2(add2(e, both(1.f)));
    const f32x2 r = pack2(rcp_fast(q.x), rcp_fast(q.y));
    const f32x2 er = mul2(e, r);
    const float2 a = unpack2(r), b = unpack2(er);
    *s = pack2(x >= 0.f ? a.x : b.x, y >= 0.f ? a.y : b.y);
    *ds = mul2(er, r);
  } else {
    const f32x2 half = exp_neg2(-0.5f * fabsf(x), -0.5f * fabsf(y));
    const f32x2 e = mul2(half, half);
    const float2 q = unpack2(add2(e, both(1.f))), h = unpack2(half);
    const float2 p = unpack2(log1p_over(e)), l = unpack2(fma2(log1p_over(e), e, pack2(x, y)));
    const float2 in = make_float2(x >= 0.f ? l.x : p.x, y >= 0.f ? l.y : p.y);   // at least log 2
    const f32x2 root = pack2(rsqrtf(in.x), rsqrtf(in.y));
    const f32x2 f = mul2(pack2(x >= 0.f ? 1.f : h.x, y >= 0.f ? 1.f : h.y), root);
    *s = mul2(f, pack2(in.x, in.y));
    *ds = mul2(mul2(f, pack2(rcp_fast(q.x), rcp_fast(q.y))), both(0.5f));
  }
}
// Where every logit is under kDeepLogit the scores are exp(h l), h = 1 (sigmoid) or 1/2
// (sqrt(softplus)), to fp32's precision, and may all be too small for fp32.  What is divided by their
// sum then takes exp(h (l - m)) in their place, m the largest logit; kDeep, e^-40, is that bound for
// the sum.  Under -745 fp64 holds no such score either, and the routing's gates are 0: so is the
// gradient.
constexpr float kDeep = 4e-18f, kDeepest = -745.f;
template <int SCORE>
constexpr float kDeepRate = SCORE == MOE_SCORE_SIGMOID ? 1.f : 0.5f;
template <int SCORE>
constexpr float kDeepLogit = SCORE == MOE_SCORE_SIGMOID ? -40.f : -80.f;

// The dense terms of a row whose scores' sum is below kDeep, by the warp: the balance term by the
// scores relative to the largest one, and zc = 2 z / T lse / sum exp(l - m) times exp(l - m).  One expert
// at a time, not in the other rows' registers: such rows are rare, and their code among the others' cost
// those 4% (896 experts, sigmoid: 54.7 us against 52.2).
template <int SCORE>
__device__ __forceinline__ void deep_row(const float* l, float* out, const float* load, int E, float aux, float m,
                                      float zc) {
  constexpr float h = kDeepRate<SCORE>;
  const int lane = threadIdx.x & 31;
  float top = -INFINITY, tot = 0.f, fp = 0.f;
#pragma unroll 1
  for (int e = lane; e < E; e += 32) top = fmaxf(top, clean_logit(l[e]));
  top = wmax(top);
  const bool some = top >= kDeepest;
  auto score = [&](float x) { return some ? unpack2(exp_neg2(h * (clean_logit(x) - top), 0.f)).x : 0.f; };
#pragma unroll 1
  for (int e = lane; e < E; e += 32) {
    const float s = score(l[e]);
    tot += s;
    fp = fmaf(load[e], s, fp);
  }
  tot = wsum(tot);
  fp = wsum(fp);
  const float inv = some ? aux * h / tot : 0.f, mean = some ? fp / tot : 0.f;
#pragma unroll 1
  for (int e = lane; e < E; e += 32) {                     // out may be l: each lane its own places
    const float x = clean_logit(l[e]);
    const float p = zc != 0.f ? zc * unpack2(exp_neg2(x - m, 0.f)).x : 0.f;
    out[e] = fmaf(inv * score(x), load[e] - mean, p);
  }
}

struct GradArgs {
  const float* logits;
  const int32_t* topk_idx;
  const float* d_gate;
  const float* load;
  float* d_logits;
  int T, E, k, renorm;
  float scale, aux, z;     // aux = aux_coef * E / T, z = 2 * z_coef / T
  int* err;
};

// What reaches every expert: nothing (only the selected ones' gradients are not zero), one dense
// term (softmax: any mix of them; others: the load-balancing loss), or the z-loss's softmax next
// to another score.
constexpr int kSparse = 0, kDense = 1, kBoth = 2;

__device__ __forceinline__ void bulk_store_row(float* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// NV: chunks of four logits a lane can hold.  BULK: rows come and go through the warp's two
// shared-memory buffers by bulk copies (rows of whole 16-byte pieces); otherwise single loads and
// stores, and one buffer to put the row together in.
// Above 512 experts the dense terms take two blocks a multiprocessor, without spills: 32768 tokens,
// 896 experts 52 us (sigmoid) and 55 (softmax), against 55 and 61 with three blocks and 80 registers;
// sqrt(softplus) 66 (80 with a square root and a division in place of one reciprocal root).
template <int NV, bool BULK, int SCORE, int TERMS>
__global__ void __launch_bounds__(32 * kGradWarps, NV <= 4 ? 4 : TERMS == kSparse ? 3 : 2)
route_grad_kernel(const GradArgs a) {
  constexpr int N = 4 * NV;
  constexpr bool SM = SCORE == MOE_SCORE_SOFTMAX;
  extern __shared__ __align__(16) uint8_t rsm[];
  __shared__ __align__(8) uint64_t s_bar[kGradWarps][2];
  __shared__ int s_abort;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int E = a.E, k = a.k;
  const uint32_t pitch = (uint32_t)(E + 3) / 4 * 16;       // bytes of a buffer
  volatile int* abort_flag = &s_abort;
  if (threadIdx.x == 0) s_abort = 0;
  __syncthreads();
  WarpRows rows;
  uint8_t* mine = rsm + (size_t)w * (BULK ? 2 : 1) * pitch;
  // the loads wait in shared memory, behind the rows
  float* s_load = reinterpret_cast<float*>(rsm + (size_t)warps * (BULK ? 2 : 1) * pitch);
  if (TERMS != kSparse && a.aux != 0.f) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) s_load[e] = __ldg(a.load + e);
    __syncthreads();
  }
  if (BULK) rows.init(s_bar[w], mine, pitch, lane);
  auto at = [&](int i) { return BULK ? 4 * (lane + 32 * (i >> 2)) + (i & 3) : lane + 32 * i; };
  auto fetch = [&](const float* p, int i, float (&f)[4], float none) {
    if constexpr (BULK) {
      float4 q = make_float4(none, none, none, none);
      if (at(i) < E) q = *reinterpret_cast<const float4*>(p + at(i));
      f[0] = q.x; f[1] = q.y; f[2] = q.z; f[3] = q.w;
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) f[c] = at(i + c) < E ? p[at(i + c)] : none;
    }
  };
  const bool gates = a.d_gate != nullptr;
  constexpr bool DENSE = TERMS != kSparse;
  constexpr bool need_p = SM ? DENSE : TERMS == kBoth;     // the full softmax
  const bool aux = DENSE && a.aux != 0.f;
  const int used = 4 * ((E + 127) / 128);                  // logits of a lane that exist (warp-uniform)
  const long long nw = (long long)gridDim.x * warps;
  const long long first = (long long)blockIdx.x * warps + w;
  unsigned it = 0, loaded = 0;                             // tokens done; rows asked for
  if (BULK && lane == 0 && first < a.T) rows.load(loaded++, a.logits + first * E);
  // a token's selection and its gates' gradients are asked for a token ahead, like its row
  int ask_sel = -1;
  float ask_u = 0.f;
  auto ask = [&](long long t) {
    if (gates && lane < k && t < a.T) {
      ask_sel = __ldg(a.topk_idx + t * k + lane);
      ask_u = __ldg(a.d_gate + t * k + lane);
    }
  };
  ask(first);
  for (long long t = first; t < a.T; t += nw, ++it) {
    const float* l = a.logits + t * E;
    float* out = reinterpret_cast<float*>(mine);           // where the row is put together
    // -------------------------------------------------- the selected experts, a lane each
    int sel = -1;
    float lf = -INFINITY, u = 0.f;
    if (gates && lane < k) {
      sel = ask_sel;
      if ((unsigned)sel >= (unsigned)E) {
        record_error(a.err, MOE_DEVERR_EXPERT_ID);
        sel = -1;
      } else {
        u = a.scale * ask_u;
      }
    }
    ask(t + nw);
    if constexpr (BULK) {
      if (!rows.wait(it, abort_flag, a.err)) break;
      out = rows.row(it);
      l = out;
      if (lane == 0 && t + nw < a.T) {
        bulk_wait_read();                                  // the row before has left the other buffer
        rows.load(loaded++, a.logits + (t + nw) * E);
      }
    }
    if (sel >= 0) lf = clean_logit(l[sel]);
    if (!(lf > -INFINITY)) u = 0.f;                        // a masked slot gives nothing, whatever d_gate holds there
    float v[N];                                            // logits; softmax: exp(l - max) further down
    if (DENSE) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        float f[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (i < used) fetch(l, i, f, -INFINITY);
#pragma unroll
        for (int c = 0; c < 4; ++c) v[i + c] = clean_logit(f[c]);
      }
    }
    float m = -INFINITY, lse = 0.f, iz = 0.f;
    if (need_p) {
#pragma unroll
      for (int i = 0; i < N; ++i) m = fmaxf(m, v[i]);
      m = wmax(m);
      if (m > -INFINITY) {
        float zs = 0.f;
        // a masked logit's exponential is 0, and so are all its terms; softmax keeps them in v
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          if ((i & ~3) >= used) continue;
          const float2 x = unpack2(exp_neg2(v[i] - m, v[i + 1] - m));
          if (SM) {
            v[i] = x.x;
            v[i + 1] = x.y;
          }
          zs += x.x + x.y;
        }
        zs = wsum(zs);
        iz = 1.f / zs;
        lse = m + logf(zs);
      } else if (SM) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.f;
      }
    }
    float dk = 0.f, p_dot = 0.f;                           // p_dot, softmax: sum_j p_{i_j} u_j
    if (gates) {
      if (SM && a.renorm) {
        const float mk = wmax(lf);
        const float ex = lf > -INFINITY ? expf(lf - mk) : 0.f;
        const float tot = wsum(ex);
        const float q = tot > 0.f ? ex / tot : 0.f;
        dk = q * (u - wsum(q * u));
      } else if (SM) {
        dk = lf > -INFINITY ? expf(lf - m) * iz * u : 0.f;
        p_dot = wsum(dk);
      } else {
        float s = 0.f, ds = 0.f;
        if (lf > -INFINITY) {
          f32x2 s2, ds2;
          score_grad2<SCORE>(lf, lf, &s2, &ds2);
          s = unpack2(s2).x;
          ds = unpack2(ds2).x;
        }
        if (a.renorm) {
          if (!__any_sync(kFull, lf > kDeepLogit<SCORE>)) {    // by every lane or none
            const float top = wmax(lf);
            if (top >= kDeepest) {
              s = unpack2(exp_neg2(kDeepRate<SCORE> * (lf - top), 0.f)).x;
              ds = kDeepRate<SCORE> * s;
            }
          }
          const float tot = wsum(s), dot = wsum(s * u);
          dk = tot > 0.f ? ds * (u - dot / tot) / tot : 0.f;
        } else {
          dk = ds * u;
        }
      }
    }
    // -------------------------------------------------- the dense terms
    float fp = 0.f, tot = 0.f;
    // the other scores' derivatives (the sigmoid's from its score, s - s^2, would lose its digits
    // where s nears 1: 2% at a logit of 12, all of them from 17 on)
    float ds_[SM ? 1 : N];
    if (aux) {
      f32x2 fp2 = both(0.f), tot2 = both(0.f);
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        if (i >= used) continue;
        float f[4];
        fetch(s_load, i, f, 0.f);
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
          const f32x2 f2 = pack2(f[c], f[c + 1]);
          if (SM) {
            fp2 = fma2(f2, pack2(v[i + c], v[i + c + 1]), fp2);
          } else {
            f32x2 s, ds;
            score_grad2<SCORE>(v[i + c], v[i + c + 1], &s, &ds);
            const float2 keep = unpack2(ds);
            ds_[SM ? 0 : i + c] = keep.x;
            ds_[SM ? 0 : i + c + 1] = keep.y;
            fp2 = fma2(f2, s, fp2);
            tot2 = add2(tot2, s);
          }
        }
      }
      fp = sum2(fp2);
      tot = sum2(tot2);
      fp = wsum(fp);
      if (SM) {
        fp *= iz;
      } else {
        tot = wsum(tot);
        fp = tot > 0.f ? fp / tot : 0.f;
      }
    }
    const float inv = !SM && aux && tot > 0.f ? a.aux / tot : 0.f;
    // softmax: dl = p (zc - p_dot + aux (f - fp)); the constant parts together
    const float flat = a.z * lse - p_dot - (SM && aux ? a.aux * fp : 0.f);
    __syncwarp();                                          // every lane has read the row
    const bool deep = !SM && aux && tot < kDeep;           // by every lane or none
    if (deep) {
      if constexpr (!SM) deep_row<SCORE>(l, out, s_load, E, a.aux, m, need_p ? iz * flat : 0.f);
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        if (i >= used || at(i) >= E) continue;
        float o[4] = {0.f, 0.f, 0.f, 0.f}, f[4] = {0.f, 0.f, 0.f, 0.f};
        if (aux) fetch(s_load, i, f, 0.f);
        if (DENSE) {
#pragma unroll
          for (int c = 0; c < 4; c += 2) {
            const f32x2 f2 = pack2(f[c], f[c + 1]);
            f32x2 g = both(0.f);
            if (SM) {
              g = aux ? fma2(both(a.aux), f2, both(flat)) : both(flat);
              g = mul2(mul2(pack2(v[i + c], v[i + c + 1]), both(iz)), g);
            } else {
              if (need_p && iz > 0.f)
                g = mul2(mul2(exp_neg2(v[i + c] - m, v[i + c + 1] - m), both(iz)), both(flat));
              if (aux) {
                const f32x2 ds = pack2(ds_[SM ? 0 : i + c], ds_[SM ? 0 : i + c + 1]);
                g = fma2(mul2(both(inv), ds), add2(f2, both(-fp)), g);
              }
            }
            const float2 h = unpack2(g);
            o[c] = h.x;
            o[c + 1] = h.y;
          }
        }
        if constexpr (BULK) {
          *reinterpret_cast<float4*>(out + at(i)) = make_float4(o[0], o[1], o[2], o[3]);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (at(i + c) < E) out[at(i + c)] = o[c];
        }
      }
    }
    __syncwarp();
    if (gates) {
      // a repeated expert's terms add up in slot order, in the lane of the last
      const bool on = sel >= 0 && lf > -INFINITY;
      const unsigned same = __match_any_sync(kFull, on ? sel : -1 - lane);
      if (__any_sync(kFull, same != 1u << lane)) {
        float sum = 0.f;
        for (int j = 0; j < k; ++j) {
          const float o = __shfl_sync(kFull, dk, j);
          if ((same >> j) & 1u) sum += o;
        }
        dk = sum;
      }
      if (on && same >> lane == 1u) out[sel] += dk;
    }
    if constexpr (BULK) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) bulk_store_row(a.d_logits + t * E, smem_u32(out), pitch);
    } else {
      __syncwarp();
      for (int e = lane; e < E; e += 32) a.d_logits[t * E + e] = out[e];
      __syncwarp();
    }
  }
  if (BULK && lane == 0) {
    rows.drain(it, loaded, a.err);                         // after a timeout: what is still in flight
    bulk_wait_all();
  }
}

template <int NV, bool BULK, int SCORE, int TERMS>
moe_status run_grad(const GradArgs& a, cudaStream_t s) {
  const int sms = num_sms();
  int warps = (a.T + sms - 1) / sms;
  if (warps > kGradWarps) warps = kGradWarps;
  constexpr size_t kMost = (size_t)kGradWarps * 2 * 4096 + 4096;   // two rows of 1024 a warp, and the loads
  static std::atomic<int> configured[kMaxDevices];
  const moe_status st = ensure_smem_limit(configured, route_grad_kernel<NV, BULK, SCORE, TERMS>, kMost);
  if (st != MOE_OK) return st;
  const size_t smem = ((size_t)warps * (BULK ? 2 : 1) + (a.aux != 0.f ? 1 : 0)) * ((a.E + 3) / 4 * 16);
  long long blocks = ((long long)a.T + warps - 1) / warps;
  const long long cap = (long long)sms * (NV <= 4 ? 4 : TERMS == kSparse ? 3 : 2);   // what a multiprocessor holds
  if (blocks > cap) blocks = cap;
  route_grad_kernel<NV, BULK, SCORE, TERMS><<<(unsigned)blocks, 32 * warps, smem, s>>>(a);
  return check_launch();
}

template <int SCORE, int TERMS>
moe_status grad_size(const GradArgs& a, bool bulk, cudaStream_t s) {
  const int nv = (a.E + 127) / 128;                        // at most 8
  if (bulk) {
    if (nv <= 1) return run_grad<1, true, SCORE, TERMS>(a, s);
    if (nv <= 2) return run_grad<2, true, SCORE, TERMS>(a, s);
    if (nv <= 4) return run_grad<4, true, SCORE, TERMS>(a, s);
    return run_grad<8, true, SCORE, TERMS>(a, s);
  }
  if (nv <= 1) return run_grad<1, false, SCORE, TERMS>(a, s);
  if (nv <= 4) return run_grad<4, false, SCORE, TERMS>(a, s);
  return run_grad<8, false, SCORE, TERMS>(a, s);
}

template <int SCORE>
moe_status grad_terms(const GradArgs& a, bool bulk, cudaStream_t s) {
  if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
    const bool dense = a.aux != 0.f || a.z != 0.f || (a.d_gate && !a.renorm);
    return dense ? grad_size<SCORE, kDense>(a, bulk, s) : grad_size<SCORE, kSparse>(a, bulk, s);
  } else {
    if (a.z != 0.f) return grad_size<SCORE, kBoth>(a, bulk, s);
    return a.aux != 0.f ? grad_size<SCORE, kDense>(a, bulk, s) : grad_size<SCORE, kSparse>(a, bulk, s);
  }
}

}  // namespace

moe_status launch_route_backward(const float* logits, const int32_t* topk_idx, const float* d_gate, int T, int E,
                                 int k, int score, int renorm, float scale, const float* load, float aux_coef,
                                 float z_coef, float* d_logits, cudaStream_t s) {
  GradArgs a{logits, topk_idx, d_gate, load, d_logits, T, E, k, renorm, scale,
             (float)((double)aux_coef * E / T), (float)(2.0 * (double)z_coef / T), err_ptr()};
  const bool bulk = E % 4 == 0 && aligned16(logits) && aligned16(d_logits);
  if (score == MOE_SCORE_SOFTMAX) return grad_terms<MOE_SCORE_SOFTMAX>(a, bulk, s);
  if (score == MOE_SCORE_SIGMOID) return grad_terms<MOE_SCORE_SIGMOID>(a, bulk, s);
  return grad_terms<MOE_SCORE_SQRT_SOFTPLUS>(a, bulk, s);
}

}  // namespace moe
