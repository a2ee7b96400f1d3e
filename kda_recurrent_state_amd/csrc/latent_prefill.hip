// Expanded latent attention over a varlen batch for gfx950: keys and values
// per head, the rotary part of the key shared by the heads.
//   s_ij = scale (q_i[:D] . k_j + q_i[D:] . kr_j),  out_i = sum_j softmax(s_i)_j v_j
// One pass over the keys with a running maximum and sum.  A wave owns 32
// queries and computes S^T = K Q^T with 32x32x16 products: a lane then holds
// one query's scores of 16 of 32 tokens, so row maxima and sums are taken in
// the lane (and its partner 32 further on), and the packed weights are already
// the right-hand operand of out^T = V^T P^T -- with the contraction in the
// order the scores lie in, which the transposed reads of V follow.
#include "internal.h"
#include "latent_common.h"

namespace kda {
namespace {

using namespace latent;

constexpr int kTile = 64;  // keys a tile

struct PrefillParams {
  const __bf16 *q, *k, *kr, *v;
  int64_t qs[2], ks[2], vs[2], krs;
  const int32_t *cu_q, *cu_k;
  __bf16* out;
  float* lse;
  int64_t T, S;
  int N, H, D, R, E, causal;
  int tiles;       // upper bound of the query tiles of a head
  float scale2;    // scale log2 e
};

__device__ __forceinline__ int64_t clamp64(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : (x > hi ? hi : x); }

// DK: D + R rounded up, EP: E rounded up, W: waves (32 queries each)
template <int DK, int EP, int W>
__global__ __launch_bounds__(W * 64, 2) void latent_prefill_kernel(PrefillParams p) {
  constexpr int KC = (DK + 63) / 64 * 8;  // 16-byte chunks of a staged key row
  constexpr int VC = EP / 8;              // and of a value row
  constexpr int KS = DK / 16;
  constexpr int MT = EP / 32;
  constexpr int kThreads = W * 64;
  constexpr int kStage = kTile * (KC + VC) * 8;
  __shared__ __attribute__((aligned(16))) __bf16 lds[2 * kStage];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ln = lane & 31, lh = lane >> 5;

  // items of one head are neighbours and run on one XCD (its L2 holds the
  // head's keys and values), the longest first
  const int64_t items = (int64_t)p.tiles * p.H, per = (items + 7) / 8;
  const int64_t item = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((int64_t)(blockIdx.x >> 3) >= per || item >= items) return;
  const int h = (int)(item / p.tiles);
  int x = p.tiles - 1 - (int)(item % p.tiles);

  // query tile x of the batch: sequence n, queries 32 W t ..
  int n = -1, t = 0;
  int64_t q0 = 0, q1 = 0;
  for (int n0 = 0; n0 < p.N; n0 += 64) {
    int64_t a = 0, b = 0;
    if (n0 + lane < p.N) {
      a = clamp64(p.cu_q[n0 + lane], 0, p.T);
      b = clamp64(p.cu_q[n0 + lane + 1], a, p.T);
    }
    const int c = (int)((b - a + 32 * W - 1) / (32 * W));
    const int incl = wave_scan(c, lane);
    const unsigned long long past = __ballot(incl > x);
    if (past) {
      const int i = __ffsll(past) - 1;
      n = n0 + i;
      t = x - __shfl(incl - c, i, 64);
      q0 = __shfl(a, i, 64);
      q1 = __shfl(b, i, 64);
      break;
    }
    x -= __shfl(incl, 63, 64);
  }
  if (n < 0) return;
  n = __builtin_amdgcn_readfirstlane(n);
  t = __builtin_amdgcn_readfirstlane(t);
  const int lq = __builtin_amdgcn_readfirstlane((int)(q1 - q0));
  const int64_t k0 = clamp64(p.cu_k[n], 0, p.S);
  const int lk = __builtin_amdgcn_readfirstlane((int)(clamp64(p.cu_k[n + 1], k0, p.S) - k0));

  const int qfirst = t * 32 * W;
  const int qi = qfirst + wave * 32 + ln;  // this lane's query
  const int64_t qrow = q0 + (qi < lq ? qi : lq - 1);
  bf16x8 qf[KS];
  {
    const __bf16* qp = p.q + qrow * p.qs[0] + h * p.qs[1];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int c = 16 * s + 8 * lh;
      bf16x8 v = {};
      if (c < p.D + p.R) v = *reinterpret_cast<const bf16x8*>(qp + c);
      qf[s] = v;
    }
  }
  // keys that this lane's query sees, and that the workgroup's last one sees
  const int sees = p.causal ? lk - (lq - 1 - qi) : lk;
  const int qlast = qfirst + 32 * W < lq ? qfirst + 32 * W : lq;
  int end = p.causal ? lk - (lq - qlast) : lk;
  end = end < 0 ? 0 : end;
  const int all_see = p.causal ? lk - (lq - 1 - (qfirst + wave * 32)) : lk;  // the wave's first query

  f32x16 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[i][j] = 0.f;
  float m = -INFINITY, l = 0.f;  // in units of scale2 s

  const int DC = p.D / 8, RC = p.R / 8, EC = p.E / 8;
  if (DC + RC < KC || EC < VC) {  // padding columns are zero from here on
    for (int i = tid; i < 2 * kStage / 8; i += kThreads) reinterpret_cast<u32x4*>(lds)[i] = u32x4{0, 0, 0, 0};
    __syncthreads();
  }
  const __bf16* kbase = p.k + k0 * p.ks[0] + h * p.ks[1];
  const __bf16* rbase = p.kr + k0 * p.krs;
  const __bf16* vbase = p.v + k0 * p.vs[0] + h * p.vs[1];

  // stages tile j (keys 64 j ..): chunk c of key row r at position c ^ (r & 7),
  // of value row r at c ^ f(r); rows behind the last key are zero
  auto vswz = [](int r) { return VC >= 16 ? (r & 7) << 1 : ((r >> 1) & 3) << 1; };
  auto stage = [&](int j, __bf16* buf) {
    __bf16* kt = buf;
    __bf16* vt = buf + kTile * KC * 8;
#pragma unroll
    for (int i = 0; i < kTile * KC / kThreads; ++i) {
      const int c0 = (i * W + wave) * 64, c = c0 + lane;
      const int r = c / KC, src = (c - r * KC) ^ (r & 7);
      const int key = j * kTile + r;
      const bool have = src < DC + RC;
      const __bf16* g = src < DC ? kbase + key * p.ks[0] + src * 8 : rbase + key * p.krs + (src - DC) * 8;
      if (have && key < lk) load_lds16(g, kt + c0 * 8);
      if (have && key >= lk) reinterpret_cast<u32x4*>(kt)[c] = u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < kTile * VC / kThreads; ++i) {
      const int c0 = (i * W + wave) * 64, c = c0 + lane;
      const int r = c / VC, src = (c - r * VC) ^ vswz(r);
      const int key = j * kTile + r;
      if (src < EC && key < lk) load_lds16(vbase + key * p.vs[0] + src * 8, vt + c0 * 8);
      if (src < EC && key >= lk) reinterpret_cast<u32x4*>(vt)[c] = u32x4{0, 0, 0, 0};
    }
  };

  const int ntiles = (end + kTile - 1) / kTile;
  if (ntiles > 0) stage(0, lds);
  for (int j = 0; j < ntiles; ++j) {
    wait_loads();
    __syncthreads();
    if (j + 1 < ntiles) stage(j + 1, lds + ((j + 1) & 1) * kStage);
    const __bf16* kt = lds + (j & 1) * kStage;
    const __bf16* vt = kt + kTile * KC * 8;

    f32x16 s[2];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[b][i] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int r = 32 * b + ln;
        const bf16x8 kf = *reinterpret_cast<const bf16x8*>(kt + (r * KC + ((2 * k + lh) ^ (r & 7))) * 8);
        s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[k], s[b], 0, 0, 0);
      }
    }
    if (j * kTile + kTile > all_see || j * kTile + kTile > lk) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int key = j * kTile + 32 * b + 8 * (i >> 2) + 4 * lh + (i & 3);
          if (key >= sees) s[b][i] = -INFINITY;
        }
    }
    float mx = s[0][0];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[b][i]);
    mx = max_halves(mx);
    const float mn = fmaxf(m, mx * p.scale2);
    const float base = mn == -INFINITY ? 0.f : mn;
    if (__any(mn > m)) {
      const float alpha = exp2_hw(m - base);
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[i] *= alpha;
      l *= alpha;
    }
    m = mn;
    // weights: bf16 for the matrix unit (the values' own type), their sum fp32
    bf16x8 pf[2][2];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float e = exp2_hw(fmaf(s[b][i], p.scale2, -base));
        l += e;
        pf[b][i >> 3][i & 7] = (__bf16)e;
      }
    // step (b, u): tokens 32 b + 16 u + {4 lh .. + 3, 8 + 4 lh .. + 3}
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const int col = 32 * i + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
          const int r0 = 32 * b + 16 * u + 4 * lh + ((lane & 15) >> 2), r1 = r0 + 8;
          const s16x4 lo = read_tr(vt + (r0 * VC + ((col >> 3) ^ vswz(r0))) * 8 + (col & 7));
          const s16x4 hi = read_tr(vt + (r1 * VC + ((col >> 3) ^ vswz(r1))) * 8 + (col & 7));
          acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(join(lo, hi), pf[b][u], acc[i], 0, 0, 0);
        }
  }

  l = sum_halves(l);
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  if (qi < lq) {
    __bf16* op = p.out + ((q0 + qi) * p.H + h) * p.E;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int col = 32 * i + 8 * g + 4 * lh;
        if (col >= p.E) continue;
        const bf16x4 o = {(__bf16)(acc[i][4 * g] * inv), (__bf16)(acc[i][4 * g + 1] * inv),
                          (__bf16)(acc[i][4 * g + 2] * inv), (__bf16)(acc[i][4 * g + 3] * inv)};
        *reinterpret_cast<bf16x4*>(op + col) = o;
      }
    if (p.lse && lh == 0) p.lse[(q0 + qi) * p.H + h] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
  }
}

template <int DK, int EP>
hipError_t launch(PrefillParams& p, hipStream_t stream) {
  constexpr int W = 4;
  p.tiles = (int)((p.T + 32 * W - 1) / (32 * W) + p.N);
  const int64_t items = (int64_t)p.tiles * p.H;
  hipLaunchKernelGGL((latent_prefill_kernel<DK, EP, W>), dim3((unsigned)((items + 7) / 8 * 8)), dim3(W * 64), 0,
                     stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_latent_prefill(const kda_latent_prefill_args_t& a, hipStream_t stream) {
  PrefillParams p;
  p.q = static_cast<const __bf16*>(a.q);
  p.k = static_cast<const __bf16*>(a.k);
  p.kr = a.R > 0 ? static_cast<const __bf16*>(a.k_rope) : p.k;
  p.v = static_cast<const __bf16*>(a.v);
  for (int i = 0; i < 2; ++i) {
    p.qs[i] = a.q_stride[i];
    p.ks[i] = a.k_stride[i];
    p.vs[i] = a.v_stride[i];
  }
  p.krs = a.R > 0 ? a.k_rope_stride : 0;
  p.cu_q = a.cu_seqlens_q;
  p.cu_k = a.cu_seqlens_k;
  p.out = static_cast<__bf16*>(a.out);
  p.lse = a.lse;
  p.T = a.T;
  p.S = a.S;
  p.N = (int)a.N;
  p.H = (int)a.H;
  p.D = (int)a.D;
  p.R = (int)a.R;
  p.E = (int)a.E;
  p.causal = a.causal != 0;
  p.scale2 = a.scale * kLog2e;
  const int64_t dk = a.D + a.R;
  if (dk <= 96 && a.E <= 64) return launch<96, 64>(p, stream);
  if (dk <= 128) return launch<128, 128>(p, stream);
  return launch<192, 128>(p, stream);
}

}  // namespace kda
