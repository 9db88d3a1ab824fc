// gka_recur, its backward and its single-token step: h_t = gamma_t h_{t-1} + beta_t x_t per channel,
// gamma = sigmoid(f), beta = 1 - gamma or 1.
//
// Bound by HBM bytes (forward 3 elements per step and channel, backward 5), so each element is read
// once. The recurrence is affine: a run of steps is the pair (A, H), A the product of its gates and
// H its result from a zero start, and (A1, H1) then (A2, H2) is (A2 A1, A2 H1 + H2). T is cut into
// segments and a segment into slices. A workgroup holds one segment of CT channels in registers, a
// thread VEC adjacent channels of one slice of L steps:
//   1. every thread reduces its slice to (A, H);
//   2. one thread per channel scans the slices' pairs in LDS and hands the segment's pair, then its
//      end state, to the workgroups of the later segments through 64-bit words in memory, and takes
//      its start from the words of the earlier ones (look-back);
//   3. every thread runs its slice from its own start and stores it.
// A word carries its own status, so no fence orders it: high half 0 = not there yet, 1 = end state,
// bit 31 set = pair (bits 0-30 are A, which is never negative), low half H or the state. The words
// and the segment counters are zeroed by a small kernel before.
// Every wait ends: the segments of a chain (batch row and channel tile) are handed out by the chain's
// counter in the order in which workgroups start, so whatever a workgroup waits for belongs to one
// that is running already, and segment 0 waits for nothing.
//
// Gates: s = exp(-|f|) / (1 + exp(-|f|)) is the smaller of gamma and 1 - gamma, to (6 + 1.25 |f|) 2^-24 of
// itself; a thread keeps v = copysign(s, f) and takes the larger one as 1 - s, rounded to nearest
// (a bias in gamma near 1 would grow with the memory's length).
//
// Infinities go as gamma h + beta x takes them. The forms above turn an infinity into NaN at the next step
// (s (x - h) + h is inf - inf), and x - h overflows where h itself does not; but what is not finite stays
// so in them. A slice whose end is not finite is therefore run again, each step that is not finite in the
// definition's form; finite channels keep their bits. A product of gates that underflows is kept above
// zero, since an infinite state survives it, while a gate of zero times infinity is NaN. The checks cost a
// finite call nothing to 2 % (8 sequences of 2048 steps by 1024 channels, slices of wider rows: 23.2 us
// with them and 22.9 without), gates of zero in every slice up to 4 %, infinite states throughout 46 to
// 69 % forward and 8 to 21 % backward.
//
// Measured (bf16): 4 sequences of 8192 steps by 2048 channels 90 us forward (4.5 TB/s) and 134 us
// backward (5.0 TB/s); one of 131072 steps by 1024 channels 180 us (4.5 TB/s) and 316 us (4.3 TB/s).
// float32: 149 us (5.4 TB/s) and 246 us (5.5 TB/s), 306 us (5.3 TB/s) and 535 us (5.0 TB/s).
// The card copies 5.1 TB/s; what is between is the start of a workgroup (counter, loads, scan,
// look-back), which only the other workgroups' loads cover: the same kernel without the look-back
// (one segment per chain) reaches 5.0 to 5.5 TB/s.
#include "gka_block.hpp"
#include "gka_rows.hpp"

namespace gka {

namespace {

// The shape of a kernel for elements T: NT threads hold SEG steps of CT channels, a thread L steps of VEC
// channels.
template <typename T, int VEC_, int CT_, int SEG_, int NT_, int WAVES_>
struct Shape {
  using Elem = T;
  static constexpr int VEC = VEC_, CT = CT_, SEG = SEG_, NT = NT_, WAVES = WAVES_;
  static constexpr int NCG = CT / VEC, NTS = NT / NCG, L = SEG / NTS;
  static_assert(NTS * L == SEG && NTS * NCG == NT, "a workgroup holds one segment");
  static_assert(SEG <= kRecurSegment, "byte offsets in a segment have 32 bits");
  // rows shorter than a vector take one channel per thread, in the same tiles and segments
  using Narrow = Shape<T, 1, CT_, SEG_, NT_, WAVES_>;
};
constexpr int kCarry = 128;  // steps between the carry's rows: every backward's segment

// Which shape a call takes. Two channels per thread fill the card with 8 waves per SIMD; in float32
// that is 8 bytes per thread and row and reaches 5.0 to 5.4 TB/s. bf16 rows of 8 bytes are 4 channels,
// at the price of 128 registers and 4 waves. Microseconds a call (side by side on one card; cards differ
// by up to 5 %), batch x steps x channels, for
// [2 channels in segments of 256 | 4 in segments of 128 | 4 in segments of 256]:
// - Forward beyond 4096 steps, the third: a chain's end states pass from segment to segment at about
//   0.1 us each, so a long sequence wants few, long segments: 1 x 131072 x 1024 [210 | 231 | 184],
//   1 x 32768 x 4096 [188 | 185 | 173]. With more tiles than CUs the second would still be ahead by 2 to
//   9 % (4 x 4352 x 2048 [56 | 53 | 58], 8 x 8192 x 2048 [191 | 164 | 169]), with few the first at first
//   (2 x 4352 x 1024 [20 | 23 | 23], 2 x 8192 x 1024 [29 | 33 | 30], 2 x 16384 x 1024 [55 | 58 | 52]).
// - Forward up to there, the second: it has two workgroups per CU, so that one loads while the other
//   scans or waits, and half-empty segments are rarer: 256 x 128 x 1024 [56 | 40 | 67],
//   64 x 512 x 1024 [51 | 52 | 55], 16 x 2048 x 1024 [53 | 50 | 52], 8 x 4096 x 2048 [104 | 92 | 98];
// - but the first for up to 2^24 elements in more than 1024 steps, a round or two of workgroups in all,
//   where more waves with half the work each are worth more: 2 x 4096 x 1024 [17.0 | 20.5 | 17.7],
//   8 x 1280 x 1024 [18.6 | 19.6 | 21.2], 4 x 1536 x 2048 [20.0 | 21.1 | 22.7]. They meet between 2^24 and
//   2^25 (4 x 2048 x 2048 [27.1 | 27.8 | 28.9], 6 x 4096 x 1024 [41.8 | 42.2 | 41.0], 12 x 2048 x 1024
//   [40.6 | 39.3 | 40.3]); at 1024 steps between 2^23 and 2^24 (8 x 1024 x 1024 [15.4 | 16.1 | 15.9],
//   8 x 1024 x 2048 [27.3 | 26.3 | 26.4]).
// - Backward [2 | 4 channels, segments of 128]: 2 (4 x 8192 x 2048 [139 | 149], 8 x 2048 x 1024
//   [42.8 | 47.0], 4 x 4096 x 1024 [43.7 | 46.9], 2 x 4096 x 1024 [24.5 | 25.9]), unless the sequence is
//   long and there are too few tiles of 64 channels to fill the card: 1 x 6144 x 1024 [23.9 | 23.4],
//   1 x 8192 x 512 [20.9 | 19.9], 1 x 131072 x 1024 [341 | 312], 1 x 131072 x 512 [204 | 162]. 2048 channels
//   in all are even from 6144 steps on (2 x 8192 x 1024 [49.0 | 47.0], 2 x 131072 x 1024 [629 | 627]), 4096
//   are not (4 x 8192 x 1024 [77 | 84]).
template <typename Fn>
inline auto with_forward(int dtype, int B, int T, int C, Fn fn) {
  if (dtype != 0) return fn(Shape<float, 2, 64, 256, 1024, 8>{});
  if (T > 4096) return fn(Shape<bf16, 4, 128, 256, 1024, 4>{});
  if (T > 1024 && (int64_t)B * C * T <= 1 << 24) return fn(Shape<bf16, 2, 64, 256, 1024, 8>{});
  return fn(Shape<bf16, 4, 128, 128, 512, 4>{});
}
template <typename Fn>
inline auto with_backward(int dtype, int B, int T, int C, Fn fn) {
  if (dtype != 0) return fn(Shape<float, 2, 64, kCarry, 1024, 8>{});
  return T > 4096 && (int64_t)B * C <= 2048 ? fn(Shape<bf16, 4, 128, kCarry, 1024, 4>{})
                                            : fn(Shape<bf16, 2, 64, kCarry, 1024, 8>{});
}

// v = copysign(min(gamma, 1 - gamma), f); f >= 0 (and +0) exactly when v's sign bit is clear
__device__ inline float gate_of(float f) { return __builtin_copysignf(sigmoids(f).small, f); }
__device__ inline bool keeps(float v) { return (int)__float_as_uint(v) >= 0; }
// v's sign in every bit, and the choice by it: one operation each and no condition mask, which the compiler
// would hold in scalar registers for every element, or wait for. In assembly, since it would make a
// comparison of them again.
__device__ inline uint32_t sign_of(float v) {
  uint32_t m;
  asm volatile("v_ashrrev_i32 %0, 31, %1" : "=v"(m) : "v"(v));
  return m;
}
__device__ inline float pick(uint32_t m, float clear, float set) {
  float r;
  asm("v_bfi_b32 %0, %1, %2, %3" : "=v"(r) : "v"(m), "v"(set), "v"(clear));
  return r;
}
__device__ inline float if_clear(uint32_t m, float a) {
  float r;
  asm("v_bfi_b32 %0, %1, 0, %2" : "=v"(r) : "v"(m), "v"(a));
  return r;
}
__device__ inline float if_set(uint32_t m, float a) { return __uint_as_float(m & __float_as_uint(a)); }
// gamma a, with one rounding; m = sign_of(v)
__device__ inline float times_gamma(float v, uint32_t m, float a) { return fmaf(-v, a, if_clear(m, a)); }
// (1 - gamma) a, with one rounding
__device__ inline float times_omg(float v, uint32_t m, float a) { return fmaf(v, a, if_set(m, a)); }
// one step: gamma h + (1 - gamma) x = the nearer of h and x plus s times the way to the other
template <bool COMP>
__device__ inline float advance(float v, uint32_t m, float h, float x) {
  return COMP ? fmaf(v, x - h, pick(m, h, x)) : times_gamma(v, m, h) + x;
}

// The same with infinities as IEEE arithmetic has them in gamma a, (1 - gamma) a and gamma h + beta x, and
// without an x - h that overflows. Steps whose result is finite have the bits of the forms above.
__device__ inline bool finite(float a) { return __builtin_isfinite(a); }
__device__ inline float rest_of(float s, float a) {  // (1 - s) a, s <= 1/2
  return fmaf(-s, fminf(fmaxf(a, -3.40282347e38f), 3.40282347e38f), a);
}
__device__ inline float times_gamma_ieee(float v, float a) {
  const float r = times_gamma(v, sign_of(v), a), s = fabsf(v);
  return finite(r) ? r : keeps(v) ? rest_of(s, a) : s * a;
}
__device__ inline float times_omg_ieee(float v, float a) {
  const float r = times_omg(v, sign_of(v), a), s = fabsf(v);
  return finite(r) ? r : keeps(v) ? s * a : rest_of(s, a);
}
template <bool COMP>
__device__ inline float advance_ieee(float v, float h, float x) {
  const float r = advance<COMP>(v, sign_of(v), h, x), s = fabsf(v);
  if (finite(r)) return r;
  if (!COMP) return times_gamma_ieee(v, h) + x;
  return keeps(v) ? fmaf(s, x, rest_of(s, h)) : fmaf(s, h, rest_of(s, x));
}
// A h + H of a run whose product of gates A may have underflown: an infinite h survives gates that are not
// zero (`zero`: one of them is)
__device__ inline float kept(float A, bool zero) { return A == 0.0f && !zero ? __uint_as_float(1u) : A; }
__device__ inline float run_end(float A, float h, float H, bool zero) {
  return fmaf(finite(h) ? A : kept(A, zero), h, H);
}

// Channels: a tile's group of VEC channels that would pass C starts at C - VEC instead, so any C >= VEC
// takes whole vectors at any alignment. Its first channels are the group's before it as well: both
// compute the same, and only the owner writes states.
template <int VEC>
__device__ inline int group_start(int nominal, int C) {
  return min(nominal, C - VEC);
}

// The rows of one segment as a buffer: `rows` rows `stride` elements apart, the last one of C
// elements. Rows from T on read as zeros and drop stores.
template <typename T>
__device__ inline __amdgpu_buffer_rsrc_t segment_buffer(const void* base, int64_t at, int64_t stride,
                                                        int rows, int C) {
  return buffer_rsrc(static_cast<const T*>(base) + at,
                     (uint32_t)((rows - 1) * stride + C) * (uint32_t)sizeof(T));
}
template <typename T, int VEC, int L>
__device__ inline void load_slice(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t stride,
                                  vec_t<T, VEC> (&v)[L]) {
#pragma unroll
  for (int l = 0; l < L; ++l)
    v[l] = buffer_load_vec<T, VEC>(r, (off + (uint32_t)l * stride) * (uint32_t)sizeof(T));
}
// The slice's gates. Steps past T keep the state (v = +0).
template <typename T, int VEC, int L>
__device__ inline void slice_gates(const vec_t<T, VEC> (&f)[L], int rows, bool tail,
                                   float (&v)[L][VEC]) {
#pragma unroll
  for (int l = 0; l < L; ++l)
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[l][i] = gate_of((float)f[l][i]);
  if (tail) {
#pragma unroll
    for (int l = 0; l < L; ++l)
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[l][i] = l < rows ? v[l][i] : 0.0f;
  }
}

// Where a thread's vectors lie: VEC channels from c0 on (its own from `nominal` on) of L steps from step t0
// of the segment on, of which `rows` steps are left before the segment's end. lane_again derives it a second
// time, so that it need not be held in registers meanwhile. (t0 < 256, and token strides below 2^22 by the
// host's check, so their products are 24-bit ones.)
struct Lane {
  int cg, ts, nominal, c0, rows;
  uint32_t t0;
};
template <typename S>
__device__ inline Lane lane_of(uint32_t tid, int tile, int C, int trows) {
  Lane q;
  q.cg = tid % S::NCG;
  q.ts = tid / S::NCG;
  q.nominal = tile * S::CT + q.cg * S::VEC;
  q.c0 = group_start<S::VEC>(q.nominal, C);
  q.t0 = (uint32_t)(q.ts * S::L);
  q.rows = trows - q.ts * S::L;
  return q;
}
template <typename S>
__device__ inline Lane lane_again(int tile, int C, int trows) {
  uint32_t tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  return lane_of<S>(tid, tile, C, trows);
}
// The gates for a rare path: what it needs of them the compiler derives there, instead of before the branch
template <int VEC, int L>
struct Again {
  float v[L][VEC];
  __device__ inline explicit Again(const float (&from)[L][VEC]) {
#pragma unroll
    for (int l = 0; l < L; ++l)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        v[l][i] = from[l][i];
        asm volatile("" : "+v"(v[l][i]));
      }
  }
};

// The slice's pairs (A, H) and, with GRAD, G. Marks the slice in the masks of the channels that have a gate
// of zero in it.
template <bool COMP, bool GRAD, typename T, int VEC, int L>
__device__ inline void slice_pairs(const float (&v)[L][VEC], const vec_t<T, VEC> (&x)[L],
                                   const vec_t<T, VEC> (&dh)[L], float (&A)[VEC], float (&H)[VEC],
                                   float (&G)[VEC], uint32_t* zeros, int ts) {
  float odd = 0.0f, least = 1.0f;  // NaN where an H or G is not finite; 0 where an A is
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    A[i] = 1.0f;
    H[i] = G[i] = 0.0f;
#pragma unroll
    for (int l = 0; l < L; ++l) {
      const uint32_t m = sign_of(v[l][i]);
      A[i] = times_gamma(v[l][i], m, A[i]);
      H[i] = advance<COMP>(v[l][i], m, H[i], (float)x[l][i]);
      if (GRAD) G[i] = fmaf(A[i], (float)dh[l][i], G[i]);
    }
    odd = fmaf(H[i], 0.0f, odd);
    if (GRAD) odd = fmaf(G[i], 0.0f, odd);
    least = fminf(least, A[i]);
  }
  if (__builtin_expect(least + odd > 0.0f, 1)) return;
  const Again<VEC, L> g(v);
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    if (A[i] == 0.0f) {
      bool zero = false;
#pragma unroll
      for (int l = 0; l < L; ++l) zero |= __float_as_uint(g.v[l][i]) == 0x80000000u;
      A[i] = kept(A[i], zero);
      if (zero) atomicOr(zeros + i, 1u << ts);
    }
    if (!finite(H[i])) {
      H[i] = 0.0f;
#pragma unroll
      for (int l = 0; l < L; ++l) H[i] = advance_ieee<COMP>(g.v[l][i], H[i], (float)x[l][i]);
    }
    if (GRAD && !finite(G[i])) {
      G[i] = 0.0f;
#pragma unroll
      for (int l = L - 1; l >= 0; --l) G[i] = times_gamma_ieee(g.v[l][i], (float)dh[l][i] + G[i]);
    }
  }
}
// (0 times an infinity is NaN)
template <int VEC>
__device__ inline bool all_finite(const float (&h)[VEC]) {
  float odd = 0.0f;
#pragma unroll
  for (int i = 0; i < VEC; ++i) odd = fmaf(h[i], 0.0f, odd);
  return odd == 0.0f;
}

__device__ inline void publish(uint64_t* word, uint32_t status, float low) {
  __hip_atomic_store(word, (uint64_t)status << 32 | __float_as_uint(low), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline void publish_pair(uint64_t* word, float A, float H) {
  publish(word, __float_as_uint(A) | 0x80000000u, H);
}
__device__ inline void publish_state(uint64_t* word, float h) { publish(word, 1u, h); }

// The state after position `at`'s predecessors, `at` the word of the position before this one: the
// nearest state among the last kLook words, carried on by the pairs after it in their order. Every
// state is the same chain of fused multiply-adds whichever state it was taken from, so results do
// not depend on timing. The words before a chain's first are another chain's (or the padding of the
// workspace): position 0 only ever holds a state, which overrides whatever came before it.
// A window of 16 words shortens the chain of one narrow sequence (a million steps of 16 channels: 238 us
// forward and 385 backward, 318 and 622 with 8) but its registers cost every other case 3 to 15 %.
constexpr int kLook = 8;
template <int CT>
__device__ inline float look_back(const uint64_t* at) {
  while (true) {
    uint64_t w[kLook];
#pragma unroll
    for (int j = 0; j < kLook; ++j)
      w[j] = __hip_atomic_load(at - j * CT, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    float h = 0.0f;
    bool have = false;
#pragma unroll
    for (int j = kLook - 1; j >= 0; --j) {
      const uint32_t hi = (uint32_t)(w[j] >> 32);
      const float low = __uint_as_float((uint32_t)w[j]);
      h = hi == 1u ? low : fmaf(__uint_as_float(hi & 0x7fffffffu), h, low);
      have = hi == 1u || (have && hi != 0u);
    }
    if (have) return h;
    __builtin_amdgcn_s_sleep(1);
  }
}

// The workgroup's chain (batch row and tile) and its position in it, from the chain's counter.
// Workgroups go round the 8 XCDs, and so do neighbouring tiles. `near`: where every chain has one XCD
// (their number is a multiple of 8), neighbours go to the same one. Tiles of rows that are no whole
// cache lines share lines, which one L2 then reads and writes once: without `near` 16 sequences of 2048
// steps by 1000 channels take 16 % more forward and 28 % more backward, 8 of 8192 by 1001 22 % and 35 %.
// With whole lines the forward is as well off dealt round (8 of 1024 by 2048 take 3 % more with `near`, 4
// of 8192 by 2048 and one of 131072 by 1024 the same), the backward is not (4 of 8192 by 2048: 14 % more
// without).
struct Spot {
  int chain, b, tile, u;
};
__device__ inline Spot take_spot(const RecurArgs& a, bool near, int* lds, uint32_t* zeros,
                                 int channels) {
  Spot p;
  const int chains = a.B * a.tiles;
  const int q = blockIdx.x % chains;
  p.chain = near && chains % 8 == 0 ? q % 8 * (chains / 8) + q / 8 : q;
  p.b = p.chain / a.tiles;
  p.tile = p.chain % a.tiles;
  p.u = 0;
  if (a.S > 1 || a.state_in) {  // (a start of zeros needs no masks)
    if (threadIdx.x < channels) zeros[threadIdx.x] = 0;
    if (a.S > 1 && threadIdx.x == 0) *lds = (int)atomicAdd(a.tickets + p.chain, 1u);
    lds_barrier();
    if (a.S > 1) p.u = __builtin_amdgcn_readfirstlane(*lds);  // uniform: scalar addresses of the segment
  }
  return p;
}

}  // namespace

__global__ __launch_bounds__(256) void recur_clear_kernel(uint4* p, int64_t n) {
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += step)
    p[i] = make_uint4(0, 0, 0, 0);
}

template <typename S, bool COMP>
__global__ __launch_bounds__(S::NT, S::WAVES) void recur_kernel(RecurArgs a) {
  using T = typename S::Elem;
  constexpr int VEC = S::VEC, L = S::L, CT = S::CT, NCG = S::NCG, NTS = S::NTS, SEG = S::SEG;
  __shared__ float sA[NTS][CT], sH[NTS][CT], start[CT];
  __shared__ int ticket;
  __shared__ uint32_t zeros[CT];  // per channel, a bit for every slice with a gate of zero
  static_assert(NTS <= 32, "one bit per slice");
  const Spot p = take_spot(a, (uint32_t)a.C * sizeof(T) % 128 != 0, &ticket, zeros, CT);
  const int tseg = p.u * SEG, trows = min(SEG, a.T - tseg);
  const Lane q = lane_of<S>(threadIdx.x, p.tile, a.C, trows);
  const int cg = q.cg, ts = q.ts, c0 = q.c0;
  // the channel that a scanning thread (of the first CT) takes, and its initial state: in its register
  // before the barrier, since the owner's wave may write the final one after it
  const int group = p.tile * CT + (int)threadIdx.x / VEC * VEC;
  const int c = group_start<VEC>(group, a.C) + threadIdx.x % VEC;
  const bool own = c >= group;
  float h0 = 0.0f;
  vec_t<T, VEC> x[L];
  float v[L][VEC];
  const auto rf = segment_buffer<T>(a.f, p.b * a.fb + tseg * a.ft, a.ft, trows, a.C);
  const auto rx = segment_buffer<T>(a.x, p.b * a.xb + tseg * a.xt, a.xt, trows, a.C);
  {
    vec_t<T, VEC> f[L];
    load_slice<T, VEC, L>(rf, __umul24(q.t0, (uint32_t)a.ft) + c0, (uint32_t)a.ft, f);
    load_slice<T, VEC, L>(rx, __umul24(q.t0, (uint32_t)a.xt) + c0, (uint32_t)a.xt, x);
    if (p.u == 0 && a.state_in && threadIdx.x < CT && group < a.C)
      h0 = a.state_in[(int64_t)p.b * a.C + c];
    slice_gates<T, VEC, L>(f, q.rows, trows < SEG, v);
  }
  {
    float A[VEC], H[VEC], none[VEC];
    slice_pairs<COMP, false, T, VEC, L>(v, x, x, A, H, none, zeros + cg * VEC, ts);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      sA[ts][cg * VEC + i] = A[i];
      sH[ts][cg * VEC + i] = H[i];
    }
  }
  asm volatile("" : "+v"(h0));
  lds_barrier();
  if (threadIdx.x < CT && group < a.C) {
    // the slices' exclusive pairs, in place, and the segment's pair (At, Ht)
    const uint32_t zero = zeros[threadIdx.x];
    float At = 1.0f, Ht = 0.0f;
#pragma unroll 16
    for (int k = 0; k < NTS; ++k) {
      const float Ak = sA[k][threadIdx.x], Hk = sH[k][threadIdx.x];
      sA[k][threadIdx.x] = At;
      sH[k][threadIdx.x] = Ht;
      Ht = fmaf(Ak, Ht, Hk);
      At *= Ak;
    }
    At = kept(At, zero != 0);
    uint64_t* word = a.words + ((int64_t)p.chain * a.S + p.u) * CT + threadIdx.x;
    const bool last = p.u == a.S - 1;
    float h = h0;
    if (p.u > 0) {
      if (!last) publish_pair(word, At, Ht);
      __atomic_signal_fence(__ATOMIC_SEQ_CST);  // the pair is on its way before the wait
      h = look_back<CT>(word - CT);
    }
    const float end = fmaf(At, h, Ht);
    if (!last)
      publish_state(word, end);
    else if (a.state_out && own)
      a.state_out[(int64_t)p.b * a.C + c] = end;
    start[threadIdx.x] = h;
    if (a.carry && own) {
      constexpr int PER = SEG / kCarry;
      const int n = (a.T + kCarry - 1) / kCarry;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        constexpr int every = kCarry / L;
        const int s = p.u * PER + j;
        if (s < n)
          a.carry[((int64_t)p.b * n + s) * a.C + c] =
              run_end(sA[j * every][threadIdx.x], h, sH[j * every][threadIdx.x],
                      (zero & ((1u << j * every) - 1)) != 0);
      }
    }
  }
  lds_barrier();
  const Lane o = lane_again<S>(p.tile, a.C, trows);
  if (o.nominal >= a.C) return;
  const auto rh = segment_buffer<T>(a.h, ((int64_t)p.b * a.T + tseg) * a.C, a.C, trows, a.C);
  // A tile of fewer than VEC channels has one group, which starts in the tile before. The state that it
  // read for that one's channels may be their final one already, so it stores its own channels alone.
  const bool crossing = VEC > 1 && p.tile * CT + VEC > a.C;
  auto store = [&](const Lane& k, int l, const float(&h)[VEC]) {
    const uint32_t at = (__umul24(k.t0, (uint32_t)a.C) + k.c0 + (uint32_t)l * (uint32_t)a.C) * (uint32_t)sizeof(T);
    if (!crossing) {
      buffer_store_vec<T, VEC>(rh, at, h);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (k.c0 + i >= k.nominal)
          buffer_store_vec<T, 1>(rh, at + (uint32_t)i * (uint32_t)sizeof(T), {h[i]});
    }
  };
  float h[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i)
    h[i] = fmaf(sA[o.ts][o.cg * VEC + i], start[o.cg * VEC + i], sH[o.ts][o.cg * VEC + i]);
#pragma unroll
  for (int l = 0; l < L; ++l) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) h[i] = advance<COMP>(v[l][i], sign_of(v[l][i]), h[i], (float)x[l][i]);
    store(o, l, h);
  }
  if (__builtin_expect(all_finite(h), 1)) return;
  // again, over what was stored: a loop that reads f and x once more, since holding them would spill
  const Lane k = lane_again<S>(p.tile, a.C, trows);
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int c = k.cg * VEC + i;
    h[i] = run_end(sA[k.ts][c], start[c], sH[k.ts][c], (zeros[c] & ((1u << k.ts) - 1)) != 0);
  }
#pragma unroll 1
  for (int l = 0; l < min(L, k.rows); ++l) {
    const uint32_t t = k.t0 + (uint32_t)l;
    const auto f = buffer_load_vec<T, VEC>(rf, (t * (uint32_t)a.ft + k.c0) * (uint32_t)sizeof(T));
    const auto xl = buffer_load_vec<T, VEC>(rx, (t * (uint32_t)a.xt + k.c0) * (uint32_t)sizeof(T));
#pragma unroll
    for (int i = 0; i < VEC; ++i) h[i] = advance_ieee<COMP>(gate_of((float)f[i]), h[i], (float)xl[i]);
    store(k, l, h);
  }
}

// Backward of one segment, the chain running from the last segment to the first. The reverse pairs
// are (A, G), G = sum_t (prod_{j <= t} gamma_j) dh_t over the run, the run's part of the gradient
// gamma q that leaves it on the left: r_left = A r_right + G. Start states come from the carry.
template <typename S, bool COMP>
__global__ __launch_bounds__(S::NT, S::WAVES) void recur_bwd_kernel(RecurArgs a) {
  using T = typename S::Elem;
  constexpr int VEC = S::VEC, L = S::L, CT = S::CT, NCG = S::NCG, NTS = S::NTS, SEG = S::SEG;
  // sA, sH, sG: the slices' pairs; then sH holds the slices' start states, and (sR, sG) the pairs of
  // the slices right of each
  __shared__ float sA[NTS][CT], sH[NTS][CT], sG[NTS][CT], sR[NTS][CT], rin[CT];
  __shared__ int ticket;
  __shared__ uint32_t zeros[CT];  // per channel, a bit for every slice with a gate of zero
  static_assert(NTS <= 32, "one bit per slice");
  const Spot p = take_spot(a, true, &ticket, zeros, CT);
  const int s = a.S - 1 - p.u;
  const int tseg = s * SEG, trows = min(SEG, a.T - tseg);
  const Lane q = lane_of<S>(threadIdx.x, p.tile, a.C, trows);
  const int cg = q.cg, ts = q.ts, c0 = q.c0;
  const int64_t dense = ((int64_t)p.b * a.T + tseg) * a.C;
  // the channel that a scanning thread takes (the first CT the gradients, the next CT the states), and
  // what it starts from
  const int k0 = threadIdx.x % CT, group = p.tile * CT + k0 / VEC * VEC;
  const int c = group_start<VEC>(group, a.C) + k0 % VEC;
  const bool real = group < a.C, own = c >= group;
  float from = 0.0f;
  vec_t<T, VEC> x[L], dh[L];
  float v[L][VEC];
  {
    vec_t<T, VEC> f[L];
    const auto rf = segment_buffer<T>(a.f, p.b * a.fb + tseg * a.ft, a.ft, trows, a.C);
    const auto rx = segment_buffer<T>(a.x, p.b * a.xb + tseg * a.xt, a.xt, trows, a.C);
    const auto rd = segment_buffer<T>(a.dh, dense, a.C, trows, a.C);
    load_slice<T, VEC, L>(rf, __umul24(q.t0, (uint32_t)a.ft) + c0, (uint32_t)a.ft, f);
    load_slice<T, VEC, L>(rx, __umul24(q.t0, (uint32_t)a.xt) + c0, (uint32_t)a.xt, x);
    load_slice<T, VEC, L>(rd, __umul24(q.t0, (uint32_t)a.C) + c0, (uint32_t)a.C, dh);
    if (real && threadIdx.x < 2 * CT) {
      if (threadIdx.x >= CT)
        from = a.carry[((int64_t)p.b * a.S + s) * a.C + c];
      else if (p.u == 0 && a.state_in)
        from = a.state_in[(int64_t)p.b * a.C + c];
    }
    slice_gates<T, VEC, L>(f, q.rows, trows < SEG, v);
  }
  {
    float A[VEC], H[VEC], G[VEC];
    slice_pairs<COMP, true, T, VEC, L>(v, x, dh, A, H, G, zeros + cg * VEC, ts);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      sA[ts][cg * VEC + i] = A[i];
      sH[ts][cg * VEC + i] = H[i];
      sG[ts][cg * VEC + i] = G[i];
    }
  }
  lds_barrier();
  if (threadIdx.x < CT && real) {
    const uint32_t zero = zeros[k0];
    float A = 1.0f, G = 0.0f;
#pragma unroll 16
    for (int k = NTS - 1; k >= 0; --k) {
      const float Ak = sA[k][k0], Gk = sG[k][k0];
      sR[k][k0] = A;
      sG[k][k0] = G;
      G = fmaf(Ak, G, Gk);
      A *= Ak;
    }
    A = kept(A, zero != 0);
    uint64_t* word = a.words + ((int64_t)p.chain * a.S + p.u) * CT + k0;
    const bool last = p.u == a.S - 1;
    float r = from;
    if (p.u > 0) {
      if (!last) publish_pair(word, A, G);
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      r = look_back<CT>(word - CT);
    }
    const float end = fmaf(A, r, G);
    if (!last)
      publish_state(word, end);
    else if (a.state_out && own)
      a.state_out[(int64_t)p.b * a.C + c] = end;
    rin[k0] = r;
  } else if (threadIdx.x >= CT && threadIdx.x < 2 * CT && real) {
    float h = from;
#pragma unroll 16
    for (int k = 0; k < NTS; ++k) {
      const float hk = h;
      h = fmaf(sA[k][k0], h, sH[k][k0]);
      sH[k][k0] = hk;
    }
  }
  lds_barrier();
  if (q.nominal >= a.C) return;
  const uint32_t first = __umul24(q.t0, (uint32_t)a.C) + c0;
  const auto rdx = segment_buffer<T>(a.h, dense, a.C, trows, a.C);
  const auto rdf = segment_buffer<T>(a.df, dense, a.C, trows, a.C);
  // runs the slice forward for its states and backward for the gradients, and stores them; whether both
  // came out finite
  auto run = [&](auto ieee, const float(&v)[L][VEC]) {
    constexpr bool IEEE = decltype(ieee)::value;
    float d[L][VEC], h[VEC], r[VEC];  // d: h_{t-1} - x, or h_{t-1}
    uint32_t m[L][VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = cg * VEC + i;
      h[i] = sH[ts][c];
      r[i] = IEEE ? run_end(sR[ts][c], rin[c], sG[ts][c], (zeros[c] >> ts >> 1) != 0)
                  : fmaf(sR[ts][c], rin[c], sG[ts][c]);
#pragma unroll
      for (int l = 0; l < L; ++l) {
        const float w = v[l][i], xv = (float)x[l][i];
        m[l][i] = sign_of(w);
        d[l][i] = COMP ? h[i] - xv : h[i];
        if (l < L - 1) h[i] = IEEE ? advance_ieee<COMP>(w, h[i], xv) : advance<COMP>(w, m[l][i], h[i], xv);
      }
    }
#pragma unroll
    for (int l = L - 1; l >= 0; --l) {
      float dx[VEC], df[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float w = v[l][i], g = (float)dh[l][i] + r[i];
        r[i] = IEEE ? times_gamma_ieee(w, g) : times_gamma(w, m[l][i], g);
        dx[i] = !COMP ? g : IEEE ? times_omg_ieee(w, g) : times_omg(w, m[l][i], g);
        // gamma (1 - gamma) = s (1 - s) for either sign of f
        df[i] = fmaf(-w, w, fabsf(w)) * (g * d[l][i]);
      }
      const uint32_t off = (first + (uint32_t)l * (uint32_t)a.C) * (uint32_t)sizeof(T);
      buffer_store_vec<T, VEC>(rdx, off, dx);
      buffer_store_vec<T, VEC>(rdf, off, df);
    }
    return all_finite(h) && all_finite(r);
  };
  if (__builtin_expect(!run(std::false_type(), v), 0)) run(std::true_type(), Again<VEC, L>(v).v);
}

// No tokens: the gradient passes through
__global__ __launch_bounds__(256) void recur_pass_kernel(const float* in, float* out, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) out[i] = in ? in[i] : 0.0f;
}

// One token: VEC channels per thread, the row's last group as in the scans (each channel is stored by
// its owner alone: the state is updated in place). 8192 sequences of 4096 channels in bf16 85 us (5.5
// TB/s); 256 of 1024 3.0 us, where any kernel takes 2.
template <typename T, int VEC, bool COMP>
__global__ __launch_bounds__(256) void recur_step_kernel(RecurArgs a) {
  const int per = (a.C + VEC - 1) / VEC;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= (int64_t)a.B * per) return;
  const int64_t b = id / per;
  const int nominal = (int)(id % per) * VEC, c = group_start<VEC>(nominal, a.C);
  const vec_t<T, VEC> x = load_vec<T, VEC>(static_cast<const T*>(a.x) + b * a.xb + c);
  const vec_t<T, VEC> f = load_vec<T, VEC>(static_cast<const T*>(a.f) + b * a.fb + c);
  float* st = a.state_out + b * a.C + c;
  T* out = static_cast<T*>(a.h) + b * a.C + c;
  const vec_t<float, VEC> h0 = load_vec<float, VEC>(st);
  float h[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const float v = gate_of((float)f[i]);
    h[i] = advance<COMP>(v, sign_of(v), h0[i], (float)x[i]);
  }
  if (__builtin_expect(!all_finite(h), 0)) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) h[i] = advance_ieee<COMP>(gate_of((float)f[i]), h0[i], (float)x[i]);
  }
  if (c == nominal) {
    store_vec<float, VEC>(st, h);
    store_vec<T, VEC>(out, h);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (c + i >= nominal) {
        st[i] = h[i];
        out[i] = from_f32<T>(h[i]);
      }
  }
}

// T / per, rounded up without passing T
static int segments(int T, int per) { return T / per + (T % per != 0); }
int recur_carry_segments(int T) { return segments(T, kCarry); }

template <typename S>
static RecurPlan plan_of(int B, int T, int C) {
  RecurPlan pl;
  pl.S = segments(T, S::SEG);
  pl.tiles = (C + S::CT - 1) / S::CT;
  const size_t chains = (size_t)B * pl.tiles;
  // words that a look-back from a chain's start may read, the words, then one counter per chain
  pl.pad = (kLook - 1) * S::CT;
  pl.words = pl.S > 1 ? chains * pl.S * S::CT : 0;
  pl.ws_bytes = pl.S > 1 ? ((pl.pad + pl.words) * 8 + chains * 4 + 255) & ~(size_t)255 : 0;
  return pl;
}
RecurPlan recur_plan(int dtype, int B, int T, int C, bool bwd) {
  auto plan = [&](auto shape) { return plan_of<decltype(shape)>(B, T, C); };
  return bwd ? with_backward(dtype, B, T, C, plan) : with_forward(dtype, B, T, C, plan);
}

static void clear_words(const RecurPlan& pl, const RecurArgs& a, hipStream_t s) {
  if (a.S == 1) return;
  const int64_t n = (int64_t)(pl.ws_bytes - pl.pad * 8) / 16, blocks = (n + 1023) / 1024;
  hipLaunchKernelGGL(recur_clear_kernel, dim3((unsigned)(blocks < 1024 ? blocks : 1024)), dim3(256), 0,
                     s, reinterpret_cast<uint4*>(a.words), n);
}

template <typename S>
static void launch_fwd(const RecurArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)a.tiles * a.B * a.S)), block(S::NT);
  if (a.complement)
    hipLaunchKernelGGL((recur_kernel<S, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((recur_kernel<S, false>), grid, block, 0, s, a);
}
hipError_t launch_recur(int dtype, const RecurPlan& pl, const RecurArgs& a, hipStream_t s) {
  clear_words(pl, a, s);
  with_forward(dtype, a.B, a.T, a.C, [&](auto shape) {
    using S = decltype(shape);
    if (a.C >= S::VEC)
      launch_fwd<S>(a, s);
    else
      launch_fwd<typename S::Narrow>(a, s);
  });
  return hipGetLastError();
}

template <typename S>
static void launch_bwd(const RecurArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)a.tiles * a.B * a.S)), block(S::NT);
  if (a.complement)
    hipLaunchKernelGGL((recur_bwd_kernel<S, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((recur_bwd_kernel<S, false>), grid, block, 0, s, a);
}
hipError_t launch_recur_bwd(int dtype, const RecurPlan& pl, const RecurArgs& a, hipStream_t s) {
  clear_words(pl, a, s);
  with_backward(dtype, a.B, a.T, a.C, [&](auto shape) {
    using S = decltype(shape);
    if (a.C >= S::VEC)
      launch_bwd<S>(a, s);
    else
      launch_bwd<typename S::Narrow>(a, s);
  });
  return hipGetLastError();
}
hipError_t launch_recur_pass(const float* in, float* out, int64_t n, hipStream_t s) {
  hipLaunchKernelGGL(recur_pass_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, in, out, n);
  return hipGetLastError();
}

template <typename T, int VEC>
static hipError_t launch_step_v(const RecurArgs& a, hipStream_t s) {
  const int64_t n = (int64_t)a.B * ((a.C + VEC - 1) / VEC);
  const dim3 grid((unsigned)((n + 255) / 256)), block(256);
  if (a.complement)
    hipLaunchKernelGGL((recur_step_kernel<T, VEC, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((recur_step_kernel<T, VEC, false>), grid, block, 0, s, a);
  return hipGetLastError();
}
hipError_t launch_recur_step(int dtype, const RecurArgs& args, hipStream_t s) {
  RecurArgs a = args;
  if (a.B == 1 || (a.xb == a.C && a.fb == a.C)) {  // dense rows are one row
    a.C *= a.B;
    a.B = 1;
  }
  if (dtype == 0) return a.C >= 8 ? launch_step_v<bf16, 8>(a, s) : launch_step_v<bf16, 1>(a, s);
  return a.C >= 4 ? launch_step_v<float, 4>(a, s) : launch_step_v<float, 1>(a, s);
}

}  // namespace gka
