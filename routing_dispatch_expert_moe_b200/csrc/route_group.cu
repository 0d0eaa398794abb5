// Group-limited top-k routing of given logits, and the gradient of a routing.
//
// Handbook news post (hub.geekagi.cn), "真正难在三个环节" item 2 (a bias for balance that only
// selects) and the quoted tweet (softmax, sigmoid, sqrt(softplus) scores); "Hugging Face 图解
// Mixture of Experts（MoE）原理、训练与推理权衡", section "什么是稀疏性？" (KeepTopK, gates) and
// the sections on the load-balancing loss and the router z-loss.
//
// moe_route_grouped.  The E experts form G groups of n = E / G.  An expert's key is its logit,
// or score + bias in fp64; a group's value is its largest key, or the sum of its two largest
// scores (+ bias).  The kept groups are the `kept` largest values, and the k largest keys of
// their experts are selected (ties to the lower index, both times).
//
// What it costs.  A token reads 4E bytes once and writes 8k; the work is the E scores, the two
// selections and the k gates, so at hundreds of experts it is bound by instruction issue.
//   - One warp per token.  A group belongs to a team of 32 / G' lanes (G' = G rounded up to a
//     power of two), so a lane finds the two largest keys of its part in registers and a few
//     shuffles finish the group.
//   - The selection runs on fp32 keys a with a known bound |a - key| <= delta.  The kept groups'
//     keys are spread evenly over the lanes through shared memory; the k-th largest of the 32
//     lane maxima is a lower bound of the k-th largest key, so everything below it (less
//     2 delta) is out.  What is left, about k to 2k experts, gets one lane each: its key in
//     fp64, and its rank by counting the larger ones.  No round per selected expert.
//   - Where fp32 cannot decide (two groups within 2 delta at the border, more than 32 experts
//     left, softmax keys within 2 delta), the warp does the token again in fp64 alone.
// So every selection is the fp64 one; the fp32 pass only discards what cannot be selected.
#include <float.h>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kGroupWarps = 8;
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
__device__ __forceinline__ double wsum_d(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ double wmax_d(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmax(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// A logit as the routing takes it: NaN counts as masked (-inf), +inf as the largest float.
__device__ __forceinline__ float clean_logit(float l) { return l > -INFINITY ? fminf(l, FLT_MAX) : -INFINITY; }

__device__ __forceinline__ double score64(double l, int score) {
  if (score == MOE_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-l));
  return sqrt(fmax(l, 0.0) + log1p(exp(-fabs(l))));
}

// log(1 + e) for 0 <= e <= 1 as 2 atanh(z), z = e / (2 + e) <= 1/3: the series in z^2 <= 1/9
// to z^15 leaves 2 z^17 / 17 < 1e-9 of it out, and keeps the relative error of a small e.
__device__ __forceinline__ float log1p_unit(float e) {
  const float z = __fdividef(e, 2.f + e), q = z * z;
  float s = 1.f / 15.f;
  s = fmaf(s, q, 1.f / 13.f);
  s = fmaf(s, q, 1.f / 11.f);
  s = fmaf(s, q, 1.f / 9.f);
  s = fmaf(s, q, 1.f / 7.f);
  s = fmaf(s, q, 1.f / 5.f);
  s = fmaf(s, q, 1.f / 3.f);
  s = fmaf(s, q, 1.f);
  return 2.f * z * s;
}
// fp32 score for discarding, with the fast exponential: its error grows with |l| (2 + 1.2 |l|
// steps), but for l < -1 the score itself falls faster, so over a row the error stays below
// the largest score times 2e-6 + 2.4e-7 |l of the largest score|.
__device__ __forceinline__ float score32(float l, int score) {
  if (score == MOE_SCORE_SIGMOID) return __fdividef(1.f, 1.f + __expf(-l));
  return sqrtf(fmaxf(l, 0.f) + log1p_unit(__expf(-fabsf(l))));
}

struct Pick {
  int idx;        // lane j < k: the j-th selected expert
  double m, z;    // softmax: largest unmasked logit and sum of exp(l - m), if they were asked for
};

// The whole selection of one token in fp64, by the warp.  Each lane keeps the keys of experts
// lane, lane + 32, ... in local memory; k rounds of an arg-max.
__device__ __noinline__ Pick route_token_fp64(const float* __restrict__ l, const float* __restrict__ bias, int E,
                                              int n, int G, int kept, int k, int score, int top2) {
  const int lane = threadIdx.x & 31;
  double key[32];
  Pick out;
  out.m = 0.0;
  out.z = 1.0;
  if (score == MOE_SCORE_SOFTMAX) {
    double m = -INFINITY, z = 0.0;
#pragma unroll 1
    for (int e = lane; e < E; e += 32) m = fmax(m, (double)clean_logit(__ldg(l + e)));
    m = wmax_d(m);
    if (m > -INFINITY) {
#pragma unroll 1
      for (int e = lane; e < E; e += 32) z += exp((double)clean_logit(__ldg(l + e)) - m);
      z = wsum_d(z);
      out.m = m;
      out.z = z;
    }
  }
  auto value = [&](int e, float lf) {                      // score (+ bias); only for lf > -inf
    const double s = score == MOE_SCORE_SOFTMAX ? exp((double)lf - out.m) / out.z : score64((double)lf, score);
    return bias ? s + (double)__ldg(bias + e) : s;
  };
#pragma unroll 1
  for (int i = 0, e = lane; e < E; ++i, e += 32) {
    const float lf = clean_logit(__ldg(l + e));
    double v = (double)lf;
    if (bias && lf > -INFINITY) {
      v = value(e, lf);
      if (v != v) v = -INFINITY;
    }
    key[i] = v;
  }
  // group values, group g's in lane g
  double mine = -INFINITY;
#pragma unroll 1
  for (int g = 0; g < G; ++g) {
    double a = -INFINITY, b = -INFINITY;                   // this lane's two largest of the group
#pragma unroll 1
    for (int i = 0, e = lane; e < E; ++i, e += 32) {
      if (e / n != g) continue;
      double v = key[i];
      if (top2 && !bias && v > -INFINITY) v = value(e, (float)v);
      if (v > a) { b = a; a = v; } else if (v > b) b = v;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const double c = __shfl_xor_sync(kFull, a, o), d = __shfl_xor_sync(kFull, b, o);
      b = fmax(fmin(a, c), fmax(b, d));
      a = fmax(a, c);
    }
    if (lane == g) mine = top2 && b > -INFINITY ? a + b : a;
  }
  int rank = 0;
#pragma unroll 1
  for (int g = 0; g < G; ++g) {
    const double v = __shfl_sync(kFull, mine, g);
    rank += v > mine || (v == mine && g < lane);
  }
  const unsigned keep = __ballot_sync(kFull, lane < G && rank < kept);
  unsigned taken = 0;
  out.idx = 0;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    double bk = -INFINITY;
    int be = 0x7fffffff;
#pragma unroll 1
    for (int i = 0, e = lane; e < E; ++i, e += 32) {
      if ((taken >> i) & 1u || !((keep >> (e / n)) & 1u)) continue;
      if (be == 0x7fffffff || key[i] > bk) { bk = key[i]; be = e; }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const double c = __shfl_xor_sync(kFull, bk, o);
      const int ce = __shfl_xor_sync(kFull, be, o);
      if (ce != 0x7fffffff && (be == 0x7fffffff || c > bk || (c == bk && ce < be))) { bk = c; be = ce; }
    }
    if (lane == j) out.idx = be;
    if ((be & 31) == lane) taken |= 1u << (be >> 5);
  }
  return out;
}

// The v-th largest (v from 1) of the 32 lanes' values: a bitonic sort, descending by lane.
__device__ __forceinline__ float kth_of_lanes(float v, int kth) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
    for (int o = size >> 1; o; o >>= 1) {
      const float c = __shfl_xor_sync(kFull, v, o);
      const bool up = ((lane & size) == 0) == ((lane & o) == 0);   // this lane keeps the larger
      v = up ? fmaxf(v, c) : fminf(v, c);
    }
  }
  return __shfl_sync(kFull, v, kth - 1);
}

struct GroupArgs {
  const float* logits;
  const float* bias;
  int32_t* topk_idx;
  float* topk_gate;
  int T, E, k, G, n, kept, team, score, top2, renorm;
  float scale;
};

// EPL: keys a lane holds of its group's part; VEC: four consecutive experts per load.
template <int EPL, bool VEC>
__global__ void __launch_bounds__(32 * kGroupWarps)
route_group_kernel(const GroupArgs a) {
  extern __shared__ float gsm[];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int E = a.E, n = a.n, k = a.k, L = a.team;
  const int pool = a.kept * n;                             // experts of the kept groups
  float* keys = gsm + (size_t)w * ((pool + 3) / 4 * 4);    // their fp32 keys, group by group
  __shared__ int s_group[kGroupWarps][32];                 // the kept groups, ascending
  __shared__ int s_cand[kGroupWarps][32];
  const int g = lane / L, tl = lane - g * L;               // this lane's group, its place in the team
  const bool in_g = g < a.G;
  const bool by_logit = !a.bias && !a.top2;                // fp32 keys are exact
  const bool need_z = a.score == MOE_SCORE_SOFTMAX && (!by_logit || !a.renorm);
  float bmax = 0.f;                                        // largest |bias|: part of the bound
  if (a.bias)
    for (int e = lane; e < E; e += 32) bmax = fmaxf(bmax, fabsf(__ldg(a.bias + e)));
  bmax = wmax(bmax);
  const long long nw = (long long)gridDim.x * kGroupWarps;
  for (long long t = (long long)blockIdx.x * kGroupWarps + w; t < a.T; t += nw) {
    const float* l = a.logits + t * E;
    // -------------------------------------------------- logits and fp32 keys
    float v[EPL];
    auto place = [&](int i) { return VEC ? 4 * (tl + L * (i >> 2)) + (i & 3) : tl + L * i; };
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < EPL; i += 4) {
        float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (in_g && place(i) < n) q = __ldg(reinterpret_cast<const float4*>(l + g * n + place(i)));
        v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) v[i] = in_g && place(i) < n ? __ldg(l + g * n + place(i)) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = clean_logit(v[i]);
    float m = -INFINITY, z = 0.f, delta = 0.f;
    if (need_z) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) m = fmaxf(m, v[i]);
      m = wmax(m);
      if (m > -INFINITY) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) z += expf(v[i] - m);
        z = wsum(z);
      }
    }
    const bool dead = need_z && !(m > -INFINITY);          // every expert masked
    if (!by_logit) {
      float smax = 0.f;
      const float iz = __fdividef(1.f, z);
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        if (v[i] > -INFINITY) {
          const float s = a.score == MOE_SCORE_SOFTMAX ? __expf(v[i] - m) * iz : score32(v[i], a.score);
          smax = fmaxf(smax, s);
          if (a.bias) {
            const float b = s + __ldg(a.bias + g * n + place(i));
            v[i] = b == b ? b : -INFINITY;
          } else {
            v[i] = s;
          }
        }
      }
      // the scores' error (see score32; where even the largest score is small, its logit is
      // about 2 log of it; softmax: the sum and its reciprocal instead), one rounding of s + b
      smax = wmax(smax);
      const float rel =
          a.score == MOE_SCORE_SOFTMAX ? 3e-6f : 2e-6f + 4.8e-7f * fmaxf(0.f, -__logf(fmaxf(smax, 1e-37f)));
      delta = rel * smax + 2.4e-7f * bmax;
    }
    // -------------------------------------------------- groups
    float g1 = -INFINITY, g2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      g2 = fmaxf(g2, fminf(g1, v[i]));
      g1 = fmaxf(g1, v[i]);
    }
    for (int o = 1; o < L; o <<= 1) {
      const float c1 = __shfl_xor_sync(kFull, g1, o), c2 = __shfl_xor_sync(kFull, g2, o);
      g2 = fmaxf(fminf(g1, c1), fmaxf(g2, c2));
      g1 = fmaxf(g1, c1);
    }
    const float gv = a.top2 && g2 > -INFINITY ? g1 + g2 : g1;
    int rank = 0;
    bool slow = false;
    for (int o = 0; o < a.G; ++o) {
      const float c = __shfl_sync(kFull, gv, o * L);
      rank += c > gv || (c == gv && o < g);
    }
    const bool keep = in_g && rank < a.kept;
    if (!by_logit && a.kept < a.G) {                       // the border must be wider than the error
      const float lo = wmax(keep ? -gv : -INFINITY), hi = wmax(in_g && !keep ? gv : -INFINITY);
      slow = !(-lo - hi > 6.f * delta + 2.4e-7f * (fabsf(lo) + fabsf(hi))) && hi > -INFINITY;
    }
    const unsigned heads = __ballot_sync(kFull, keep && tl == 0);
    const int order = __popc(heads & ((1u << (g * L)) - 1u));   // this group's place among the kept
    // -------------------------------------------------- the kept groups' keys, spread evenly
    if (a.top2 && !a.bias) {
      // groups by scores, experts by logit: the logits again
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (keep && place(i) < n) v[i] = clean_logit(__ldg(l + g * n + place(i)));
      delta = 0.f;
    }
    __syncwarp();                                          // the previous token's keys are read
    if (keep) {
      if (tl == 0) s_group[w][order] = g;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (place(i) < n) keys[order * n + place(i)] = v[i];
    }
    __syncwarp();
    float best = -INFINITY;
    for (int p = lane; p < pool; p += 32) best = fmaxf(best, keys[p]);
    float tau = kth_of_lanes(best, k);
    auto count = [&](float th) {
      int c = 0;
      for (int p = lane; p < pool; p += 32) c += keys[p] >= th;
      return (int)__reduce_add_sync(kFull, (unsigned)c);
    };
    // the keys not below the threshold, in index order; the first 32 get a lane each
    auto compact = [&]() {
      const float th = tau - 2.f * delta - (delta > 0.f ? 2.4e-7f * fabsf(tau) : 0.f);
      int c = 0;
      for (int p0 = 0; p0 < pool; p0 += 32) {
        const int p = p0 + lane;
        const bool in = p < pool && keys[p] >= th;
        const unsigned b = __ballot_sync(kFull, in);
        const int at = c + __popc(b & ((1u << lane) - 1u));
        if (in && at < 32) s_cand[w][at] = p;
        c += __popc(b);
      }
      return c;
    };
    int c = compact();
    if (c > 32 && tau > -INFINITY) {
      // the lane maxima bound it too loosely (many selected, or unlucky): halve the way from
      // the bound to the largest key, keeping at least k keys above it
      float lo = tau, hi = wmax(best);
      for (int it = 0; it < 24; ++it) {
        const float mid = 0.5f * lo + 0.5f * hi;
        const int above = count(mid);
        if (above >= k) lo = mid; else hi = mid;
        if (above >= k && above <= 32) break;
      }
      tau = lo;
      __syncwarp();
      c = compact();
    }
    __syncwarp();
    slow = slow || !(tau > -INFINITY) || c > 32 || c < k;
    // -------------------------------------------------- exact order of what is left
    Pick pick;
    pick.idx = 0;
    pick.m = (double)m;
    pick.z = (double)z;
    if (!slow) {
      int e = 0;
      double key = -INFINITY;
      if (lane < c) {
        const int p = s_cand[w][lane];
        const int o = p / n;
        e = s_group[w][o] * n + (p - o * n);
        if (!a.bias)
          key = (double)clean_logit(__ldg(l + e));
        else if (a.score == MOE_SCORE_SOFTMAX)
          key = (double)keys[p];                           // checked against delta below
        else
          key = score64((double)clean_logit(__ldg(l + e)), a.score) + (double)__ldg(a.bias + e);
      }
      int r = 0;
      bool near = false;
      const double gap = a.bias && a.score == MOE_SCORE_SOFTMAX ? 2.0 * (double)delta : -1.0;
      for (int j = 0; j < c; ++j) {
        const double o = __shfl_sync(kFull, key, j);
        // candidates are in index order, so a lower lane is a lower index
        r += o > key || (o == key && j < lane);
        near = near || (j != lane && fabs(o - key) <= gap);
      }
      slow = __any_sync(kFull, near && lane < c);
      if (lane < c && r < k) s_cand[w][r] = e;             // every lane has read its candidate
      __syncwarp();
      if (lane < k) pick.idx = s_cand[w][lane];
    }
    if (slow) pick = route_token_fp64(l, a.bias, E, n, a.G, a.kept, k, a.score, a.top2);
    // -------------------------------------------------- gates (fp64, rounded once)
    const bool act = lane < k;
    const float lf = act ? clean_logit(__ldg(l + pick.idx)) : -INFINITY;
    double s = 0.0;
    if (a.score == MOE_SCORE_SOFTMAX) {
      if (a.renorm) {
        const double mm = wmax_d((double)lf);
        s = lf > -INFINITY ? exp((double)lf - mm) : 0.0;
      } else {
        s = lf > -INFINITY && !dead ? exp((double)lf - pick.m) / pick.z : 0.0;
      }
    } else if (lf > -INFINITY) {
      s = score64((double)lf, a.score);
    }
    if (a.renorm) {
      const double tot = wsum_d(s);
      s = tot > 0.0 ? s / tot : 0.0;
    }
    if (act) {
      a.topk_idx[t * k + lane] = pick.idx;
      a.topk_gate[t * k + lane] = (float)(s * (double)a.scale);
    }
    __syncwarp();
  }
}

template <int EPL, bool VEC>
moe_status run_group(const GroupArgs& a, cudaStream_t s) {
  const size_t smem = (size_t)kGroupWarps * ((a.kept * a.n + 3) / 4 * 4) * sizeof(float);   // at most 32 KB
  long long blocks = ((long long)a.T + kGroupWarps - 1) / kGroupWarps;
  const long long cap = (long long)num_sms() * 8;
  if (blocks > cap) blocks = cap;
  route_group_kernel<EPL, VEC><<<(unsigned)blocks, 32 * kGroupWarps, smem, s>>>(a);
  return check_launch();
}

}  // namespace

moe_status launch_route_grouped(const float* logits, int T, int E, int k, int n_groups, int groups_kept,
                                int group_score, int score, int renorm, float scale, const float* bias,
                                int32_t* topk_idx, float* topk_gate, cudaStream_t s) {
  GroupArgs a{logits, bias, topk_idx, topk_gate, T, E, k, n_groups, E / n_groups, groups_kept, 0, score,
              group_score == MOE_GROUP_TOP2, renorm, scale};
  int p2 = 1;
  while (p2 < n_groups) p2 <<= 1;
  a.team = 32 / p2;
  const bool vec = a.n % 4 == 0 && aligned16(logits);
  const int per = vec ? (a.n / 4 + a.team - 1) / a.team * 4 : (a.n + a.team - 1) / a.team;   // at most 64
  if (vec) {
    if (per <= 4) return run_group<4, true>(a, s);
    if (per <= 8) return run_group<8, true>(a, s);
    if (per <= 16) return run_group<16, true>(a, s);
    if (per <= 32) return run_group<32, true>(a, s);
    return run_group<64, true>(a, s);
  }
  if (per <= 4) return run_group<4, false>(a, s);
  if (per <= 8) return run_group<8, false>(a, s);
  if (per <= 16) return run_group<16, false>(a, s);
  if (per <= 32) return run_group<32, false>(a, s);
  return run_group<64, false>(a, s);
}

}  // namespace moe
