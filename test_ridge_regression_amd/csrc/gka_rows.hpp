// Device-side building blocks of the block operators: vector loads, the gate's activation, sums
// over a team of lanes (gfx950).
#pragma once

#include <type_traits>

#include "gka_common.hpp"

namespace gka {

template <typename T, int VEC>
using vec_t = T __attribute__((ext_vector_type(VEC)));

// VEC elements at any address that is a multiple of the element's size: one load or store of the
// vector's width (gfx950 takes unaligned global accesses).
template <typename T, int VEC>
__device__ inline vec_t<T, VEC> load_vec(const T* p) {
  vec_t<T, VEC> v;
  __builtin_memcpy(&v, p, sizeof v);
  return v;
}
template <typename T, int VEC>
__device__ inline void store_vec(T* p, const float (&v)[VEC]) {
  vec_t<T, VEC> o;
#pragma unroll
  for (int i = 0; i < VEC; ++i) o[i] = from_f32<T>(v[i]);
  __builtin_memcpy(p, &o, sizeof o);
}

// Rows of D elements held by a team of lanes: `lanes` lanes, NV vectors of VEC <= D elements each.
// Vector j of a lane holds the elements from (lane + j lanes) VEC on. The vector that would pass the
// row's end starts at D - VEC instead, so a row of any length and alignment takes whole vectors. Its
// first `skip` elements are also the vector's before it: both compute them, sums count them once, and
// both store the same values (skip = VEC: the row has ended before this vector).
template <int VEC, int NV>
struct RowPart {
  int start[NV], skip[NV];
  __device__ inline RowPart(int lane, int lanes, int D) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (lane + j * lanes) * VEC;
      start[j] = min(c, D - VEC);
      skip[j] = min(c - start[j], VEC);
    }
  }
};
// Element `off` past a uniform `base`, by a 32-bit byte offset. (The empty asm keeps the compiler from
// widening the offset to 64 bits outside a loop: a load or store then takes the base from scalar
// registers and one vector register, where it would add 64-bit pairs and hold them.)
template <typename T>
__device__ inline T* at_offset(T* base, uint32_t off) {
  using Byte = typename std::conditional<std::is_const<T>::value, const char, char>::type;
  uint32_t bytes = off * (uint32_t)sizeof(T);
  asm volatile("" : "+v"(bytes));
  return reinterpret_cast<T*>(reinterpret_cast<Byte*>(base) + bytes);
}
template <typename T, int VEC, int NV>
__device__ inline void load_row(const T* base, uint32_t off, const RowPart<VEC, NV>& p,
                                vec_t<T, VEC> (&v)[NV]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) v[j] = load_vec<T, VEC>(at_offset(base, off + (uint32_t)p.start[j]));
}
// The sum over a lane's elements of f(j, i), each counted once in the row
template <int VEC, int NV, typename F>
__device__ inline float row_sum(const RowPart<VEC, NV>& p, const F& f) {
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) v += f(j, i);
    if (p.skip[j]) {
      v = 0.0f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) v += i >= p.skip[j] ? f(j, i) : 0.0f;
    }
    s += v;
  }
  return s;
}
// `alias`: an output of the call is read from the same memory, so an element must be stored by its owner
// alone, who has read it before any of it is stored
template <typename T, int VEC, int NV>
__device__ inline void store_row(T* base, uint32_t off, const RowPart<VEC, NV>& p, int j,
                                 const float (&v)[VEC], bool alias = false) {
  T* at = at_offset(base, off + (uint32_t)p.start[j]);
  if (p.skip[j] == 0 || (!alias && p.skip[j] < VEC)) {
    store_vec<T, VEC>(at, v);
  } else if (alias) {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (i >= p.skip[j]) at[i] = from_f32<T>(v[i]);
  }
}
// Float32 weights of the row, `fill` without any
template <int VEC, int NV>
__device__ inline void load_weights(const float* w, const RowPart<VEC, NV>& p, float fill,
                                    float (&v)[NV][VEC]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    vec_t<float, VEC> x = (vec_t<float, VEC>)fill;
    if (w) x = load_vec<float, VEC>(w + p.start[j]);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[j][i] = x[i];
  }
}

// VEC elements `off` bytes into a buffer: zeros past its end, with no branch around the load (a
// branch would make every load wait for the one before). VEC divides what the buffer holds.
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
template <typename T, int VEC>
__device__ inline vec_t<T, VEC> buffer_load_vec(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  constexpr int N = sizeof(T) * VEC;
  static_assert(N == 2 || N == 4 || N == 8 || N == 16, "one load");
  if constexpr (N == 2) {
    return __builtin_bit_cast(vec_t<T, VEC>, __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0));
  } else if constexpr (N == 4) {
    return __builtin_bit_cast(vec_t<T, VEC>, __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
  } else if constexpr (N == 8) {
    return __builtin_bit_cast(vec_t<T, VEC>, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
  } else {
    return __builtin_bit_cast(vec_t<T, VEC>, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
  }
}
// and the store, dropped past the end
template <typename T, int VEC>
__device__ inline void buffer_store_vec(__amdgpu_buffer_rsrc_t r, uint32_t off,
                                        const float (&v)[VEC]) {
  constexpr int N = sizeof(T) * VEC;
  static_assert(N == 2 || N == 4 || N == 8 || N == 16, "one store");
  vec_t<T, VEC> o;
#pragma unroll
  for (int i = 0; i < VEC; ++i) o[i] = from_f32<T>(v[i]);
  if constexpr (N == 2) {
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, o), r, off, 0, 0);
  } else if constexpr (N == 4) {
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned int, o), r, off, 0, 0);
  } else if constexpr (N == 8) {
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2_t, o), r, off, 0, 0);
  } else {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, o), r, off, 0, 0);
  }
}
// The byte offset of a lane's vector j in its row as a buffer; past any row's end for a vector without
// elements of its own, whose store is dropped
template <typename T, int VEC, int NV>
__device__ inline uint32_t row_offset(const RowPart<VEC, NV>& p, int j) {
  return p.skip[j] < VEC ? (uint32_t)p.start[j] * (uint32_t)sizeof(T) : 0xfffffff0u;
}

// sigmoid(|g|) and sigmoid(-|g|) from e = exp(-|g|) by the hardware's exp2 and reciprocal (1 ulp each):
// 1 / (1 + e) and e / (1 + e). Infinite g give 1, 0. The rounded argument |g| log2(e) of exp2 leaves the
// smaller one a relative error of up to (6 + 1.25 |g|) 2^-24: below 1e-6 up to |g| = 8, 6e-6 at 80.
// (Splitting the argument would save it at two more operations per element; where |g| is large the smaller
// one is small beside what it is added to.)
struct Sigmoids {
  float large, small;
};
__device__ inline Sigmoids sigmoids(float g) {
  const float e = __builtin_amdgcn_exp2f(fabsf(g) * -1.44269504f);
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  return {r, e * r};
}

// The gate's activation: silu (g sigmoid(g)) or sigmoid; 1 without a gate
enum class Act { kSilu = 0, kSigmoid = 1, kNone = 2 };
__device__ inline float gate_act(float g, Act a) {
  const Sigmoids p = sigmoids(g);
  const float s = g >= 0.0f ? p.large : p.small;
  return a == Act::kNone ? 1.0f : (a == Act::kSilu ? g : 1.0f) * s;
}
// and its slope: sigmoid' = s (1 - s) is the product of the two sigmoids, silu' = s + g s (1 - s)
__device__ inline float gate_act(float g, Act a, float& slope) {
  const Sigmoids p = sigmoids(g);
  const float s = g >= 0.0f ? p.large : p.small, t = p.large * p.small;
  slope = a == Act::kSilu ? fmaf(g, t, s) : t;
  return a == Act::kNone ? 1.0f : (a == Act::kSilu ? g : 1.0f) * s;
}

// Sums over the lanes of a team, in every lane of it, always in the same order. TEAM = 1 .. 64: that
// many consecutive lanes of a wave, by DPP moves within 16 lanes and the row swaps beyond. TEAM = 0:
// the whole workgroup of up to 16 waves; red is LDS for 16 float2, and a caller alternates between
// two of them from one sum to the next (a sum's barrier keeps its writers from the readers of the
// sum before the last).
template <int CTRL>
__device__ inline float dpp_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL,
                                                                   0xf, 0xf, true));
}
template <int LANES>
__device__ inline float lanes_sum(float v) {
  if constexpr (LANES >= 2) v = dpp_add<0xB1>(v);    // lane ^ 1
  if constexpr (LANES >= 4) v = dpp_add<0x4E>(v);    // lane ^ 2
  if constexpr (LANES >= 8) v = dpp_add<0x141>(v);   // lane 7 - i of 8
  if constexpr (LANES >= 16) v = dpp_add<0x140>(v);  // lane 15 - i of 16
  if constexpr (LANES >= 32) {
    float a = v, b = v;
    swap_rows16(a, b);
    v = a + b;
  }
  if constexpr (LANES >= 64) {
    float a = v, b = v;
    swap_rows32(a, b);
    v = a + b;
  }
  return v;
}
template <int TEAM>
__device__ inline float2 team_sum(float2 v, float2* red) {
  constexpr int LANES = TEAM ? TEAM : kWave;
  v = make_float2(lanes_sum<LANES>(v.x), lanes_sum<LANES>(v.y));
  if constexpr (TEAM == 0) {
    const int lane = threadIdx.x % kWave;
    if (lane == 0) red[threadIdx.x / kWave] = v;
    lds_barrier();
    const int w = lane % 16;
    v = w < (int)blockDim.x / kWave ? red[w] : make_float2(0.0f, 0.0f);
    v = make_float2(lanes_sum<16>(v.x), lanes_sum<16>(v.y));
  }
  return v;
}
template <int TEAM>
__device__ inline float team_sum(float v, float2* red) {
  constexpr int LANES = TEAM ? TEAM : kWave;
  v = lanes_sum<LANES>(v);
  if constexpr (TEAM == 0) {
    const int lane = threadIdx.x % kWave;
    if (lane == 0) red[threadIdx.x / kWave].x = v;
    lds_barrier();
    const int w = lane % 16;
    v = lanes_sum<16>(w < (int)blockDim.x / kWave ? red[w].x : 0.0f);
  }
  return v;
}

}  // namespace gka
