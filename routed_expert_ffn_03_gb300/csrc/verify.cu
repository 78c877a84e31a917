// verify.cu - which drafted tokens stand, and the token drawn after them.
//
// Draft i with token t stands iff u_i q_i(t) < p_i(t); the token after the last that stands
// is drawn by inverting the running sum of max(p - q, 0) (or of p, when every draft stands).
// A weight x (p - q rounded to fp32, by 2^-24 of itself at most) is carried as the integer
// x 2^60, rounded, in 64 bits, so sums are exact and the same in any order, and the token is the least v with
// cum(v) > floor(u total): an integer comparison, with u a 64-bit fraction.
//
// Only the row that decides is read, once: a cluster of S blocks takes a sequence, each warp a contiguous run of
// the vocabulary in 16-byte words of p (q starts at another offset in its 16 bytes when V is odd, so its words are
// put together from two loads).  The warps' sums are scanned over the cluster through distributed
// shared memory, and the one warp whose run holds the threshold walks it again (from L2).  Bound: memory, with the
// arithmetic close behind (about 14 instructions an element).
#include "common.cuh"
#include "grouped.h"
#include "grouped_mma.cuh"
#include "verify.h"

namespace moe {

namespace {

constexpr int VF_THREADS = 256;
constexpr int VF_WARPS = VF_THREADS / 32;
constexpr int VF_MAX_CLUSTER = 8;
constexpr int VF_DEPTH = 4;
constexpr int VF_STEP = 32 + 34;                       // 16-byte words of a step (33 of q, and one to keep 32 bytes)
constexpr int VF_SMEM = VF_WARPS * VF_DEPTH * VF_STEP * 16;
typedef unsigned long long u64;

// clamped to [0, 1]; max with NaN gives the other operand, 0
__device__ __forceinline__ float clamp01(float x) { return fminf(fmaxf(x, 0.f), 1.f); }
template <int DT>
__device__ __forceinline__ float load_prob(const char* p, long long i) {
  if (DT == GT_FP32) return __ldg(reinterpret_cast<const float*>(p) + i);
  const uint16_t b = __ldg(reinterpret_cast<const uint16_t*>(p) + i);
  return DT == GT_BF16 ? bf16_bits_to_float(b) : __half2float(__ushort_as_half(b));
}
// the elements of a 16-byte word
template <int DT>
struct Word {
  static constexpr int EL = DT == GT_FP32 ? 4 : 2, N = 16 / EL;
  float x[N];
  __device__ __forceinline__ void decode(const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (DT == GT_FP32) {
        x[i] = __uint_as_float(w[i]);
      } else if (DT == GT_BF16) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        const __half2 h = *reinterpret_cast<const __half2*>(&w[i]);
        x[2 * i] = __low2float(h);
        x[2 * i + 1] = __high2float(h);
      }
    }
  }
};

// max(a - b, 0) clamped to [0, 1], NaN as 0: one instruction
__device__ __forceinline__ float sub_sat(float a, float b) {
  float r;
  asm("sub.sat.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void copy16(uint4* dst, const uint4* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// pairs of fp32, one instruction for both
__device__ __forceinline__ u64 pair(float lo, float hi) {
  u64 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ u64 pair_add(u64 a, u64 b) {
  u64 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ u64 pair_fma(u64 a, u64 b, u64 c) {
  u64 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// The sum of x 2^60, each rounded to an integer, over several x in [0, 1]: 1 + x has x 2^23 rounded in its low bits, and what
// is left over, signed, gives the next 23 bits in the same way, and the last 14.  7 instructions a pair and 3
// additions an element.  (The conversion instruction to 64 bits runs at the FP64 rate, low on this part, shifts take 9
// instructions of the integer pipe, at half the rate, and additions rounded to zero do not come in pairs.)
struct Sum60 {
  uint32_t a = 0, b = 0, c = 0;
  __device__ __forceinline__ void add(float x0, float x1) {
    const u64 one = pair(1.f, 1.f), minus = pair(-1.f, -1.f), mid = pair(1.5f, 1.5f), x = pair(x0, x1);
    const u64 h = pair_add(x, one);
    const u64 r = pair_fma(pair_add(h, minus), minus, x);                                    // exact, 2^-24 at most
    const u64 m = pair_fma(r, pair(8388608.f, 8388608.f), mid);
    const u64 l = pair_fma(pair_add(m, pair(-1.5f, -1.5f)), pair(-1.1920928955078125e-7f, -1.1920928955078125e-7f), r);   // 2^-47
    const u64 n = pair_fma(l, pair(137438953472.f, 137438953472.f), mid);
    a += (uint32_t)h + (uint32_t)(h >> 32);
    b += (uint32_t)m + (uint32_t)(m >> 32);
    c += (uint32_t)n + (uint32_t)(n >> 32);
  }
  // of n elements (up to 256: the signed middle parts fill 32 bits)
  __device__ __forceinline__ u64 total(uint32_t n) const {
    return ((u64)(a - n * 0x3f800000u) << 37) + (u64)((long long)(int)(b - n * 0x3fc00000u) << 14) +
           (u64)(long long)(int)(c - n * 0x3fc00000u);
  }
};
__device__ __forceinline__ u64 fixed60(float x) {
  Sum60 s;
  s.add(x, 0.f);
  return s.total(2);
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 w = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += w;
  }
  return v;
}

// The row that decides: weights max(p - q, 0), or p without q, `hot` (a one-hot draft, or -1) left out.
template <int DT>
struct Row {
  typedef Word<DT> W;
  const char *p, *q;
  int V, hot;
  int head, words;    // elements before the first word, whole 16-byte words of p after
  int shift;          // bytes by which q's counterpart of a word of p is off a boundary

  __device__ __forceinline__ void set(const char* p_, const char* q_, int hot_, int V_) {
    p = p_;
    q = q_;
    hot = hot_;
    V = V_;
    head = min((int)((16 - ((uintptr_t)p & 15)) & 15) / W::EL, V);
    words = (V - head) / W::N;
    shift = q ? (int)(((uintptr_t)q + (uintptr_t)head * W::EL) & 15) : 0;
    if (shift) {   // the two words of q around p's first and last word reach past the row: those go by elements
      const bool any = words >= 2;
      head += any ? W::N : 0;
      words = any ? words - 2 : 0;
    }
  }
  __device__ __forceinline__ u64 one(int v) const {
    const float a = load_prob<DT>(p, v);
    return v == hot ? 0 : fixed60(sub_sat(a, q ? load_prob<DT>(q, v) : 0.f));
  }
  // 16 bytes from `shift` on of two neighbouring words (the branch is the same for the whole row)
  __device__ __forceinline__ uint4 align(const uint4& lo, const uint4& hi) const {
    const int by = 8 * (shift & 3);
    auto cut = [&](uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e) {
      return make_uint4(__funnelshift_r(a, b, by), __funnelshift_r(b, c, by), __funnelshift_r(c, d, by), __funnelshift_r(d, e, by));
    };
    if (shift < 4) return cut(lo.x, lo.y, lo.z, lo.w, hi.x);
    if (shift < 8) return cut(lo.y, lo.z, lo.w, hi.x, hi.y);
    if (shift < 12) return cut(lo.z, lo.w, hi.x, hi.y, hi.z);
    return cut(lo.w, hi.x, hi.y, hi.z, hi.w);
  }
  __device__ __forceinline__ const uint4* p_at(int c) const {
    return reinterpret_cast<const uint4*>(p + (size_t)head * W::EL) + c;
  }
  __device__ __forceinline__ const uint4* q_at(int c) const {   // its first word, `shift` bytes early
    return reinterpret_cast<const uint4*>(q + (size_t)head * W::EL - shift) + c;
  }
  // the weights of word c from its 16 bytes of p and of q
  template <bool Q>
  __device__ __forceinline__ W weights(int c, const uint4& pw, const uint4& qw) const {
    W a, b;
    a.decode(pw);
    if (Q) b.decode(qw);
    const int skip = hot - head - c * W::N;
#pragma unroll
    for (int i = 0; i < W::N; ++i) a.x[i] = Q ? sub_sat(a.x[i], b.x[i]) : i == skip ? 0.f : sub_sat(a.x[i], 0.f);
    return a;
  }
  template <bool Q>
  __device__ __forceinline__ W word(int c) const {
    uint4 qw = make_uint4(0, 0, 0, 0);
    if (Q) qw = shift ? align(__ldg(q_at(c)), __ldg(q_at(c) + 1)) : __ldg(q_at(c));
    return weights<Q>(c, __ldg(p_at(c)), qw);
  }
  static __device__ __forceinline__ u64 sum_of(const W& w) {
    Sum60 s;
#pragma unroll
    for (int i = 0; i < W::N; i += 2) s.add(w.x[i], w.x[i + 1]);
    return s.total(W::N);
  }
  // Words [c0, c1) by one warp, through its ring of VF_DEPTH steps of 32 words of p and 33 of q: the copies in flight need no
  // registers.
  template <bool Q>
  __device__ __forceinline__ u64 sum_words(int c0, int c1, int lane, uint4* ring) const {
    const int steps = (c1 - c0 + 31) / 32;
    auto issue = [&](int i) {
      const int c = c0 + i * 32 + lane;
      uint4* at = ring + (i % VF_DEPTH) * VF_STEP + lane;
      if (i < steps && c < c1) {
        copy16(at, p_at(c));
        if (Q) {
          copy16(at + 32, q_at(c));
          if (shift && (lane == 31 || c == c1 - 1)) copy16(at + 33, q_at(c) + 1);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < VF_DEPTH - 1; ++i) issue(i);
    u64 sum = 0;
    for (int i = 0; i < steps; ++i) {
      issue(i + VF_DEPTH - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(VF_DEPTH - 1) : "memory");
      __syncwarp();
      const int c = c0 + i * 32 + lane;
      const uint4* at = ring + (i % VF_DEPTH) * VF_STEP + lane;
      if (c < c1) {
        uint4 qw = make_uint4(0, 0, 0, 0);
        if (Q) qw = shift ? align(at[32], at[33]) : at[32];
        sum += sum_of(weights<Q>(c, at[0], qw));
      }
      __syncwarp();   // the step's slot is written again from the next round on
    }
    return sum;
  }
  // A warp's walk to the least element with run + cumulative weight > thr.  One step of up to 32 elements, or words, from
  // `at`: advances run, returns the element or -1 (the same in every lane).
  __device__ __forceinline__ int step(bool is_words, int at, int end, u64 thr, u64& run, int lane) const {
    u64 w[W::N];
    u64 s = 0;
#pragma unroll
    for (int i = 0; i < W::N; ++i) w[i] = 0;
    const int me = at + lane;
    if (me < end) {
      if (!is_words) s = w[0] = one(me);
      else {
        const W x = q ? word<true>(me) : word<false>(me);
#pragma unroll
        for (int i = 0; i < W::N; ++i) s += w[i] = fixed60(x.x[i]);
      }
    }
    const u64 cum = run + warp_scan(s, lane);
    const unsigned hit = __ballot_sync(0xffffffffu, cum > thr);
    int found = -1;
    if (hit) {
      u64 c = cum - s;
      int k = 0;
#pragma unroll
      for (int i = 0; i < W::N; ++i) {
        c += w[i];
        if (c <= thr) k = i + 1;
      }
      found = __shfl_sync(0xffffffffu, is_words ? head + me * W::N + k : me, __ffs(hit) - 1);
    }
    run = __shfl_sync(0xffffffffu, cum, 31);
    return found;
  }
  // Words [c0, c1): first the sums of AHEAD steps whose loads are all in flight, then the one step that holds it.
  template <bool Q>
  __device__ __forceinline__ int walk_words(int c0, int c1, u64 thr, u64& run, int lane) const {
    constexpr int AHEAD = 4;
    for (int c = c0; c < c1; c += 32 * AHEAD) {
      u64 s[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) s[i] = c + 32 * i + lane < c1 ? sum_of(word<Q>(c + 32 * i + lane)) : 0;
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const u64 sum = warp_sum(s[i]);
        if (run + sum > thr) return step(true, c + 32 * i, c1, thr, run, lane);
        run += sum;
      }
    }
    return -1;
  }
};

__device__ __forceinline__ void st_cluster64(uint32_t addr, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

template <int DT>
__global__ void __launch_bounds__(VF_THREADS, 4) verify_kernel(VerifyArgs a, int S) {
  __shared__ u64 part[VF_WARPS];
  __shared__ u64 block_sum[2][VF_MAX_CLUSTER];   // by attempt and rank: every block writes its sum to all
  extern __shared__ uint4 rings[];
  constexpr int EL = Word<DT>::EL;
  const int b = blockIdx.x / S, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = S > 1 ? (int)cluster_rank() : 0;
  const char* p = static_cast<const char*>(a.p) + (long long)b * a.p_seq * EL;
  const char* q = a.q ? static_cast<const char*>(a.q) + (long long)b * a.q_seq * EL : nullptr;

  if (S > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // this block has started

  // lane i: draft i (every warp alike, so nothing is passed between them)
  const int L = a.lengths ? min(max(__ldg(a.lengths + b), 0), a.D) : a.D;
  int tok = -1;
  bool stands = true;
  if (lane < a.D) tok = __ldg(a.draft + (long long)b * a.D + lane);
  const float u = lane <= a.D ? clamp01(__ldg(a.u + (long long)b * (a.D + 1) + lane)) : 0.f;
  if (lane < L) {
    stands = false;
    if (tok >= 0 && tok < a.V) {
      const float pv = clamp01(load_prob<DT>(p + lane * a.p_row * EL, tok));
      const float qv = q ? clamp01(load_prob<DT>(q + lane * a.q_row * EL, tok)) : 1.f;
      const float uq = u * qv;   // and what its rounding left: the comparison is exact
      stands = uq < pv || (uq == pv && __fmaf_rn(u, qv, -uq) < 0.f);
    }
  }
  const unsigned no = __ballot_sync(0xffffffffu, !stands);
  const int r = no ? __ffs(no) - 1 : L;
  const int rejected = __shfl_sync(0xffffffffu, tok, r & 31);
  const float uf = __shfl_sync(0xffffffffu, u, a.D);
  const u64 U = uf >= 1.f ? ~0ull : __float2ull_rz(uf * 18446744073709551616.f);

  Row<DT> row;
  row.set(p + r * a.p_row * EL, r < L && q ? q + r * a.q_row * EL : nullptr, r < L && !q ? rejected : -1, a.V);
  const int W = S * VF_WARPS, me = rank * VF_WARPS + warp;
  const int c0 = (int)((long long)row.words * me / W), c1 = (int)((long long)row.words * (me + 1) / W);
  const int tail = row.head + row.words * Word<DT>::N;   // the first element behind the words
  uint4* ring = rings + warp * VF_DEPTH * VF_STEP;
  bool drawn = false;
  for (int attempt = 0; attempt < 2; ++attempt) {
    u64 sum = row.q ? row.template sum_words<true>(c0, c1, lane, ring) : row.template sum_words<false>(c0, c1, lane, ring);
    if (me == 0 && lane < row.head) sum += row.one(lane);
    if (me == W - 1 && tail + lane < a.V) sum += row.one(tail + lane);
    sum = warp_sum(sum);
    if (attempt) __syncthreads();   // part has been read
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    u64 before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < VF_WARPS; ++w) {
      if (w == warp) before = total;
      total += part[w];
    }
    if (S > 1) {
      if (attempt == 0) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // and so have the others
      if ((int)threadIdx.x < S) st_cluster64(map_rank(smem_u32(&block_sum[attempt][rank]), threadIdx.x), total);
      cluster_sync_all();   // after it nothing is read from another block: a block may end when it has no more to do
      const u64 s = lane < S ? block_sum[attempt][lane] : 0;
      const u64 inc = warp_scan(s, lane);
      total = __shfl_sync(0xffffffffu, inc, 31);
      before += __shfl_sync(0xffffffffu, inc - s, rank);
    }
    if (total) {
      const u64 thr = __umul64hi(U, total);   // floor(u total) < total
      if (before <= thr && thr < before + sum) {
        u64 run = before;
        int v = -1;
        if (me == 0) v = row.step(false, 0, row.head, thr, run, lane);
        if (v < 0)
          v = row.q ? row.template walk_words<true>(c0, c1, thr, run, lane) : row.template walk_words<false>(c0, c1, thr, run, lane);
        if (v < 0) v = row.step(false, tail, a.V, thr, run, lane);
        if (lane == 0) a.tokens[(long long)b * (a.D + 1) + r] = v;
      }
      drawn = true;
      break;
    }
    if (!row.q && row.hot < 0) break;   // p itself is empty
    row.q = nullptr;                    // nothing left of the residual: draw from p
    row.hot = -1;
  }
  if (rank == 0 && warp == 0 && lane <= a.D) {
    int* out = a.tokens + (long long)b * (a.D + 1);
    if (lane < r) out[lane] = tok;
    else if (lane > r || !drawn) out[lane] = -1;
    if (lane == 0) a.accepted[b] = r;
  }
}

template <int DT>
cudaError_t launch_as(const VerifyArgs& a, int S, cudaStream_t s) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)a.B * S);
  c.blockDim = dim3(VF_THREADS);
  c.dynamicSmemBytes = VF_SMEM;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = S;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, verify_kernel<DT>, a, S);
}

}  // namespace

cudaError_t verify_set_attributes() {
  cudaError_t e = cudaFuncSetAttribute(verify_kernel<GT_FP32>, cudaFuncAttributeMaxDynamicSharedMemorySize, VF_SMEM);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(verify_kernel<GT_BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, VF_SMEM);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(verify_kernel<GT_FP16>, cudaFuncAttributeMaxDynamicSharedMemorySize, VF_SMEM);
  return e;
}

cudaError_t launch_verify(const VerifyArgs& a, int num_sms, cudaStream_t s) {
  // Blocks to a sequence: four to an SM in all, so that one streams while others wait (a block is a chain of waits: drafts,
  // sums, scan, walk), with a few words for every lane.  256 sequences of 129281 in 1 / 2 / 4 / 8 blocks each:
  // 77 / 51 / 43 / 44 us; 64 sequences: 58 / 33 / 22 / 19 us; blocks of 512 threads: 53 / 48 / 50 / 66 us.
  int S = 1;
  while (S < VF_MAX_CLUSTER && (long long)a.B * S < 4 * num_sms && a.V >= 2048 * S) S *= 2;
  if (a.dtype == GT_FP32) return launch_as<GT_FP32>(a, S, s);
  return a.dtype == GT_BF16 ? launch_as<GT_BF16>(a, S, s) : launch_as<GT_FP16>(a, S, s);
}

}  // namespace moe
