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
// put together from two).  The blocks' sums are scanned over the cluster through distributed
// shared memory, and the block whose share holds the threshold searches the run of the warp that does, all threads at
// once (from L2; by that warp alone it took a quarter of the kernel's time).  Bound: 256 sequences of 129281 in bf16 with q
// take 33 us, of which reading the rows is 17 at the memory's rate (116 MB); the rest is a block's chain of waits.
#include "common.cuh"
#include "grouped.h"
#include "grouped_mma.cuh"
#include "verify.h"

namespace moe {

namespace {

constexpr int VF_MAX_CLUSTER = 8;
constexpr int VF_DEPTH = 3;
constexpr int VF_STEP = 64;                            // 16-byte words of p in a step, two a lane
constexpr int VF_SLOT = VF_STEP + VF_STEP + 2;         // with q's (one more where q is off a boundary, one to keep 32 bytes)
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
  // 16 bytes from `shift` on of two neighbouring words; SH: shift / 4
  template <int SH>
  __device__ __forceinline__ uint4 align(const uint4& lo, const uint4& hi) const {
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    if (W::EL == 4) return make_uint4(w[SH], w[SH + 1], w[SH + 2], w[SH + 3]);
    const int by = 8 * (shift & 3);
    return make_uint4(__funnelshift_r(w[SH], w[SH + 1], by), __funnelshift_r(w[SH + 1], w[SH + 2], by),
                      __funnelshift_r(w[SH + 2], w[SH + 3], by), __funnelshift_r(w[SH + 3], w[SH + 4], by));
  }
  __device__ __forceinline__ uint4 align(const uint4& lo, const uint4& hi) const {
    if (shift < 4) return align<0>(lo, hi);
    if (shift < 8) return align<1>(lo, hi);
    return shift < 12 ? align<2>(lo, hi) : align<3>(lo, hi);
  }
  __device__ __forceinline__ const uint4* p_at(int c) const {
    return reinterpret_cast<const uint4*>(p + (size_t)head * W::EL) + c;
  }
  __device__ __forceinline__ const uint4* q_at(int c) const {   // its first word, `shift` bytes early
    return reinterpret_cast<const uint4*>(q + (size_t)head * W::EL - shift) + c;
  }
  // the weights of a word from its 16 bytes of p and of q
  template <bool Q>
  static __device__ __forceinline__ W weights(const uint4& pw, const uint4& qw) {
    W a, b;
    a.decode(pw);
    if (Q) b.decode(qw);
#pragma unroll
    for (int i = 0; i < W::N; ++i) a.x[i] = sub_sat(a.x[i], Q ? b.x[i] : 0.f);
    return a;
  }
  template <bool Q>
  __device__ __forceinline__ W word(int c) const {
    uint4 qw = make_uint4(0, 0, 0, 0);
    if (Q) qw = shift ? align(__ldg(q_at(c)), __ldg(q_at(c) + 1)) : __ldg(q_at(c));
    W a = weights<Q>(__ldg(p_at(c)), qw);
    const int skip = hot - head - c * W::N;
#pragma unroll
    for (int i = 0; i < W::N; ++i)
      if (!Q && i == skip) a.x[i] = 0.f;
    return a;
  }
  static __device__ __forceinline__ u64 sum_of(const W& w) {
    Sum60 s;
#pragma unroll
    for (int i = 0; i < W::N; i += 2) s.add(w.x[i], w.x[i + 1]);
    return s.total(W::N);
  }
  // Words [c0, c1) by one warp, through its ring of VF_DEPTH steps: the copies in flight need no registers.  Q: with q, SH:
  // shift / 4, -1 where q stands on a boundary too.  `hot` is left in.
  template <bool Q, int SH>
  __device__ __forceinline__ u64 sum_words(int c0, int c1, int lane, uint4* ring) const {
    const int n = c1 - c0, full = n / VF_STEP, rest = n % VF_STEP, steps = full + (rest != 0);
    const uint4 *ps = p_at(c0) + lane, *qs = Q ? q_at(c0) + lane : nullptr;
    ring += lane;
    auto issue = [&](int i, int slot) {
      uint4* at = ring + slot * VF_SLOT;
      if (i < full) {
        copy16(at, ps);
        copy16(at + 32, ps + 32);
        if (Q) {
          copy16(at + VF_STEP, qs);
          copy16(at + VF_STEP + 32, qs + 32);
          if (SH >= 0 && lane == 31) copy16(at + VF_STEP + 33, qs + 33);
        }
        ps += VF_STEP;
        if (Q) qs += VF_STEP;
      } else if (i < steps) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (lane + 32 * j < rest) {
            copy16(at + 32 * j, ps + 32 * j);
            if (Q) copy16(at + VF_STEP + 32 * j, qs + 32 * j);
            if (SH >= 0 && (lane == 31 || lane + 32 * j == rest - 1)) copy16(at + VF_STEP + 32 * j + 1, qs + 32 * j + 1);
          }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto add_word = [&](const uint4* at, Sum60& s) {
      uint4 qw = make_uint4(0, 0, 0, 0);
      if (Q) qw = SH >= 0 ? align<SH < 0 ? 0 : SH>(at[VF_STEP], at[VF_STEP + 1]) : at[VF_STEP];
      const W x = weights<Q>(at[0], qw);
#pragma unroll
      for (int i = 0; i < W::N; i += 2) s.add(x.x[i], x.x[i + 1]);
    };
    issue(0, 0);
    issue(1, 1);
    u64 sum = 0;
    Sum60 s;
    constexpr int RUN = 256 / (2 * W::N);   // steps whose sums fit 32 bits
    int slot = 0;
    for (int i = 0; i < full; ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(VF_DEPTH - 2) : "memory");
      __syncwarp();   // every lane's copies are there, and the slot written next has been read
      issue(i + 2, slot ? slot - 1 : 2);
      const uint4* at = ring + slot * VF_SLOT;
      add_word(at, s);
      add_word(at + 32, s);
      if (i % RUN == RUN - 1) {
        sum += s.total(256);
        s = Sum60();
      }
      slot = slot == 2 ? 0 : slot + 1;
    }
    sum += s.total((uint32_t)(full % RUN) * 2 * W::N);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (lane + 32 * j < rest) {
        Sum60 t;
        add_word(ring + slot * VF_SLOT + 32 * j, t);
        sum += t.total(W::N);
      }
    __syncwarp();   // the ring may be written again
    return sum;
  }
  // one warp's sum of its words
  __device__ __forceinline__ u64 sum_of_run(int c0, int c1, int lane, uint4* ring) const {
    if (!q) {
      u64 sum = sum_words<false, -1>(c0, c1, lane, ring);
      const int at = hot - head;
      if (hot >= 0 && at >= c0 * W::N && at < c1 * W::N && lane == 0) sum -= fixed60(sub_sat(load_prob<DT>(p, hot), 0.f));
      return sum;
    }
    switch (shift ? shift >> 2 : -1) {
      case 0: return sum_words<true, DT == GT_FP32 ? -1 : 0>(c0, c1, lane, ring);
      case 1: return sum_words<true, 1>(c0, c1, lane, ring);
      case 2: return sum_words<true, 2>(c0, c1, lane, ring);
      case 3: return sum_words<true, 3>(c0, c1, lane, ring);
      default: return sum_words<true, -1>(c0, c1, lane, ring);
    }
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
  // The least element of words [c0, c1) with run + cumulative weight > thr, by the whole block: each thread sums a few
  // neighbouring words, and the warp of the one that holds it steps through those.  -1 in the other warps; run advances to
  // the sum behind the words, and is > thr in all of them if the element is among the words.  A run of more than 8 words
  // a thread is first cut down to the warp's share that holds it.
  template <bool Q, int WARPS>
  __device__ __forceinline__ int search(int c0, int c1, u64 thr, u64& run, int lane, u64* part) const {
    const int warp = threadIdx.x >> 5;
    while (c1 - c0 > 8 * 32 * WARPS) {
      const int len = c1 - c0, a0 = c0 + (int)((long long)len * warp / WARPS), a1 = c0 + (int)((long long)len * (warp + 1) / WARPS);
      u64 mine = 0;
#pragma unroll 4
      for (int w = a0 + lane; w < a1; w += 32) mine += sum_of(word<Q>(w));
      mine = warp_sum(mine);
      if (lane == 0) part[warp] = mine;
      __syncthreads();
      int hit = 0;
      while (hit < WARPS && run + part[hit] <= thr) run += part[hit++];
      __syncthreads();   // part has been read
      if (hit == WARPS) return -1;
      c1 = c0 + (int)((long long)len * (hit + 1) / WARPS);
      c0 += (int)((long long)len * hit / WARPS);
    }
    const int n = c1 - c0, per = (n + WARPS * 32 - 1) / (WARPS * 32);
    const int w0 = c0 + min((int)threadIdx.x * per, n), w1 = min(w0 + per, c1);
    u64 mine = 0;
#pragma unroll 4
    for (int w = w0; w < w1; ++w) mine += sum_of(word<Q>(w));
    const u64 inc = warp_scan(mine, lane);
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    u64 before = run;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w == warp) before = run;
      run += part[w];
    }
    before += inc - mine;
    const unsigned hit = __ballot_sync(0xffffffffu, before <= thr && thr < before + mine);
    int found = -1;
    if (hit) {
      const int l = __ffs(hit) - 1;
      u64 at = __shfl_sync(0xffffffffu, before, l);
      const int end = __shfl_sync(0xffffffffu, w1, l);
      for (int w = __shfl_sync(0xffffffffu, w0, l); w < end && found < 0; w += 32) found = step(true, w, end, thr, at, lane);
    }
    return found;
  }
};

__device__ __forceinline__ void st_cluster64(uint32_t addr, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

template <int DT, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) verify_kernel(VerifyArgs a, int S) {
  constexpr int VF_WARPS = THREADS / 32;
  __shared__ u64 part[VF_WARPS], found_part[VF_WARPS];
  __shared__ u64 block_sum[2][VF_MAX_CLUSTER];   // by attempt and rank: every block writes its sum to all
  extern __shared__ uint4 rings[];
  constexpr int EL = Word<DT>::EL;
  const int b = blockIdx.x / S, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = S > 1 ? (int)cluster_rank() : 0;
  const char* p = static_cast<const char*>(a.p) + (long long)b * a.p_seq * EL;
  const char* q = a.q ? static_cast<const char*>(a.q) + (long long)b * a.q_seq * EL : nullptr;

  if (S > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // this block has started

  pdl_wait();   // (the next kernel is not let in early: its blocks would crowd on the SMs that have room)
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
      stands = (double)u * (double)qv < (double)pv;   // exact: 48 bits, and no product below fp64's range
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
  uint4* ring = rings + warp * VF_DEPTH * VF_SLOT;
  bool drawn = false;
  for (int attempt = 0; attempt < 2; ++attempt) {
    u64 sum = row.sum_of_run(c0, c1, lane, ring);
    if (me == 0 && lane < row.head) sum += row.one(lane);
    if (me == W - 1 && tail + lane < a.V) sum += row.one(tail + lane);
    sum = warp_sum(sum);
    if (attempt) __syncthreads();   // part has been read
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    u64 block = 0, before = 0;   // the block's sum, and the blocks' before it
#pragma unroll
    for (int w = 0; w < VF_WARPS; ++w) block += part[w];
    u64 total = block;
    if (S > 1) {
      if (attempt == 0) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // and so have the others
      if ((int)threadIdx.x < S) st_cluster64(map_rank(smem_u32(&block_sum[attempt][rank]), threadIdx.x), block);
      cluster_sync_all();   // after it nothing is read from another block: a block may end when it has no more to do
      const u64 s = lane < S ? block_sum[attempt][lane] : 0;
      const u64 inc = warp_scan(s, lane);
      total = __shfl_sync(0xffffffffu, inc, 31);
      before = __shfl_sync(0xffffffffu, inc - s, rank);
    }
    if (total) {
      const u64 thr = __umul64hi(U, total);   // floor(u total) < total
      if (before <= thr && thr < before + block) {   // the same in the whole block
        u64 run = before;
        int hit = 0;   // the warp whose run holds it
        while (hit < VF_WARPS - 1 && run + part[hit] <= thr) run += part[hit++];
        const int h = rank * VF_WARPS + hit;
        const int h0 = (int)((long long)row.words * h / W), h1 = (int)((long long)row.words * (h + 1) / W);
        int v = -1;
        if (h == 0) v = row.step(false, 0, row.head, thr, run, lane);
        if (v < 0) {
          v = row.q ? row.template search<true, VF_WARPS>(h0, h1, thr, run, lane, found_part)
                    : row.template search<false, VF_WARPS>(h0, h1, thr, run, lane, found_part);
          if (run <= thr) v = row.step(false, tail, a.V, thr, run, lane);
        }
        if (lane == 0 && v >= 0) a.tokens[(long long)b * (a.D + 1) + r] = v;   // (each warp that has it has the same)
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

constexpr int verify_smem(int threads) { return threads / 32 * VF_DEPTH * VF_SLOT * 16; }

template <int DT, int THREADS>
cudaError_t launch_as(const VerifyArgs& a, int S, cudaStream_t s) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)a.B * S);
  c.blockDim = dim3(THREADS);
  c.dynamicSmemBytes = verify_smem(THREADS);
  c.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = S;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 2;
  return cudaLaunchKernelEx(&c, verify_kernel<DT, THREADS>, a, S);
}
template <int THREADS>
cudaError_t launch_type(const VerifyArgs& a, int S, cudaStream_t s) {
  if (a.dtype == GT_FP32) return launch_as<GT_FP32, THREADS>(a, S, s);
  return a.dtype == GT_BF16 ? launch_as<GT_BF16, THREADS>(a, S, s) : launch_as<GT_FP16, THREADS>(a, S, s);
}

}  // namespace

cudaError_t verify_set_attributes() {
  auto set = [](void (*kernel)(VerifyArgs, int)) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, verify_smem(256));
  };
  cudaError_t e = set(verify_kernel<GT_FP32, 256>);
  if (e == cudaSuccess) e = set(verify_kernel<GT_BF16, 256>);
  if (e == cudaSuccess) e = set(verify_kernel<GT_FP16, 256>);
  return e;
}

cudaError_t launch_verify(const VerifyArgs& a, int num_sms, cudaStream_t s) {
  // Blocks to a sequence: 8, while that makes no more than two blocks an SM, or leaves each 60000 bytes of p: small shares
  // have more waits (drafts, sums, scan, search) to an element, large ones end less evenly.  In 1 / 2 / 4 / 8 blocks each,
  // us: 64 sequences of 129281 in bf16 21 / 14 / 12.1 / 12.3; 256 35 / 36 / 33 / 37; 512 65 / 54 / 54 / 66; 256 of 32000
  // 10.4 / 12.0 / 14.9 / 21.2.
  const int el = a.dtype == GT_FP32 ? 4 : 2;
  int S = VF_MAX_CLUSTER;
  while (S > 1 && (a.V < 1024 * S || ((long long)a.B * S > 2 * num_sms && (long long)a.V * el < 60000ll * S))) S /= 2;
  // Many short sequences: of blocks of 128 threads twice as many stand on an SM.  2048 of 3000 in bf16 15 and 23 us, of 12000
  // 29 and 35, of 24000 49 and 46; 608 of 12000 14 and 11.
  if (a.B > 4 * num_sms && (long long)a.V * el < 40000) return launch_type<128>(a, 1, s);
  return launch_type<256>(a, S, s);
}

}  // namespace moe
