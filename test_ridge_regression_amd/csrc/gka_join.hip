// gka_join and its backward: the end of a block fused with the next block's norm.
//   u = y rstd(y) w_post act(gate),  r' = res + alpha scale u,  n = r' rstd(r') w_pre
//
// Bound by HBM bytes (forward 5 elements per channel, backward 8). A token's row is held in the
// registers of one team of lanes (RowPlan with one head), so every operand is read once and the two
// norms cost one sum over the team each. The backward computes u and r' again from the forward's
// inputs instead of reading a rounded r'; then
//   G = dr' + rstd' (dn w_pre - rh c2), rh = r' rstd', c2 = mean(dn w_pre rh)
//   du = alpha scale G,  e = du w_post act(gate),  dy = rstd_y (e - yh c1), c1 = mean(e yh)
// which is three dependent sums per row. Weight gradients are summed as in the gated norm: per lane
// over the team's tokens, the workgroup's teams in LDS, the workgroups by column_sums_kernel.
//
// Measured, calls one after another: 16384 bf16 tokens of 4096 channels 122 us forward (5.5 TB/s) and
// 213 us backward (5.0 TB/s; the card copies 5.1), 7 of which are the weight gradients' second kernel;
// with a float32 stream, 32768 tokens of 1024 channels 84 us (5.6 TB/s) and 154 us (4.8 TB/s). Slower: the
// bf16 backward beyond 4096 channels (8192: 3.6 TB/s, 4.3 with a float32 stream; 5120: 3.4; 4099: 2.6),
// where one workgroup per CU has nothing loaded ahead, the narrower widths as many waves as they need and
// not what the CU could hold; and odd bf16 widths that leave lanes or waves idle (333: 4.3 TB/s forward,
// 3.5 backward).
#include "gka_block.hpp"
#include "gka_rows.hpp"

namespace gka {

// A team of TEAM lanes (0: the workgroup) holds one row; a workgroup's teams take adjacent rows, and
// it strides over the rows by `step` (uniform), so that a lane's offsets from the start of its
// workgroup's rows never change.
struct JoinPlace {
  int lane, team;
  int64_t t0, step;
};
template <int TEAM>
__device__ inline JoinPlace join_place(const RowPlan& pl) {
  JoinPlace p;
  p.lane = TEAM ? threadIdx.x % (TEAM ? TEAM : 1) : threadIdx.x;
  p.team = TEAM ? threadIdx.x / (TEAM ? TEAM : 1) : 0;
  p.t0 = (int64_t)blockIdx.x * pl.tt;
  p.step = (int64_t)gridDim.x * pl.tt;
  return p;
}

template <typename R, typename T, int VEC, int TEAM, int NV>
__global__ __launch_bounds__(TEAM ? 256 : 1024) void join_kernel(JoinArgs a, RowPlan pl) {
  __shared__ float2 red[2][16];
  const JoinPlace p = join_place<TEAM>(pl);
  const RowPart<VEC, NV> rp(p.lane, TEAM ? TEAM : blockDim.x, a.C);
  const float inv_c = 1.0f / (float)a.C;
  const Act act = a.gate ? (Act)a.act : Act::kNone;
  const bool post = a.w_post != nullptr, pre = a.w_pre != nullptr;

  float wp[NV][VEC], sc[NV][VEC], wn[NV][VEC];
  load_weights<VEC, NV>(a.w_post, rp, 1.0f, wp);
  load_weights<VEC, NV>(a.scale, rp, 1.0f, sc);
  load_weights<VEC, NV>(a.w_pre, rp, 1.0f, wn);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) sc[j][i] *= a.alpha;
  // in place, what a lane reads of another's elements may be the new stream already: only the owners store
  const bool in_place = a.res_out == a.res;
  // without a gate its loads repeat y's
  const T* gate = static_cast<const T*>(a.gate ? a.gate : a.y);
  const int64_t gate_stride = a.gate ? a.gate_stride : a.y_stride;
  const uint32_t team = (uint32_t)p.team, oo = team * (uint32_t)a.C;
  for (int64_t t0 = p.t0; t0 < a.rows; t0 += p.step) {
    if (TEAM && t0 + p.team >= a.rows) break;
    vec_t<R, VEC> r[NV];
    vec_t<T, VEC> y[NV], g[NV];
    load_row<T, VEC, NV>(static_cast<const T*>(a.y) + t0 * a.y_stride, team * (uint32_t)a.y_stride,
                         rp, y);
    load_row<T, VEC, NV>(gate + t0 * gate_stride, team * (uint32_t)gate_stride, rp, g);
    load_row<R, VEC, NV>(static_cast<const R*>(a.res) + t0 * a.res_stride,
                         team * (uint32_t)a.res_stride, rp, r);
    float ry = 1.0f;
    if (post) {
      const float m =
          row_sum<VEC, NV>(rp, [&](int j, int i) { return (float)y[j][i] * (float)y[j][i]; });
      ry = rsqrtf(team_sum<TEAM>(m, red[0]) * inv_c + a.eps);
    }
    float ro[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float u = (float)y[j][i] * ry * wp[j][i] * gate_act((float)g[j][i], act);
        ro[j][i] = fmaf(sc[j][i], u, (float)r[j][i]);
      }
      store_row<R, VEC, NV>(static_cast<R*>(a.res_out) + t0 * a.C, oo, rp, j, ro[j], in_place);
    }
    float rr = 0.0f;
    if (pre) {
      const float m2 = row_sum<VEC, NV>(rp, [&](int j, int i) { return ro[j][i] * ro[j][i]; });
      rr = rsqrtf(team_sum<TEAM>(m2, red[1]) * inv_c + a.eps);
    }
    // with both norms their sums alternate between two buffers; with one, its buffer is written
    // again in the next row
    if (TEAM == 0 && !(post && pre)) lds_barrier();
    if (!pre) continue;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float o[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] = ro[j][i] * rr * wn[j][i];
      store_row<T, VEC, NV>(static_cast<T*>(a.n) + t0 * a.C, oo, rp, j, o, in_place);
    }
  }
}

// The backward's operands of one row (without a gate, or without w_pre and so dn, those loads repeat
// y's and do not count)
template <typename R, typename T, int VEC, int NV>
struct JoinBwdRow {
  vec_t<R, VEC> r[NV], dr[NV];
  vec_t<T, VEC> y[NV], g[NV], dn[NV];
  __device__ inline void load(const JoinArgs& a, int64_t t0, uint32_t team,
                              const RowPart<VEC, NV>& rp) {
    const T* yb = static_cast<const T*>(a.y);
    const T* gb = static_cast<const T*>(a.gate ? a.gate : a.y);
    const T* nb = static_cast<const T*>(a.dn ? a.dn : a.y);
    const int64_t gs = a.gate ? a.gate_stride : a.y_stride, ns = a.dn ? a.C : a.y_stride;
    load_row<T, VEC, NV>(yb + t0 * a.y_stride, team * (uint32_t)a.y_stride, rp, y);
    load_row<T, VEC, NV>(gb + t0 * gs, team * (uint32_t)gs, rp, g);
    load_row<R, VEC, NV>(static_cast<const R*>(a.res) + t0 * a.res_stride,
                         team * (uint32_t)a.res_stride, rp, r);
    load_row<T, VEC, NV>(nb + t0 * ns, team * (uint32_t)ns, rp, dn);
    load_row<R, VEC, NV>(static_cast<const R*>(a.dres_out) + t0 * a.C, team * (uint32_t)a.C, rp, dr);
  }
};

// What the compiler derives from a row after this it derives again, instead of holding conversions and
// gates in registers across the sums. Two vectors per lane then fit 128 registers but for 2 with a float32
// stream and 6 in float32: 4096 rows of 8192 channels, bf16 with a float32 stream, take 170 us (270 with
// 46 spilled registers). (Loads of the next row during a row, which one vector per lane has, spill again
// and cost 25 to 50 % here.)
template <typename V, int NV>
__device__ inline void renew(V (&v)[NV]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    struct Words {
      uint32_t w[sizeof(V) / 4];
    } u = __builtin_bit_cast(Words, v[j]);
#pragma unroll
    for (size_t k = 0; k < sizeof(V) / 4; ++k) asm volatile("" : "+v"(u.w[k]));
    v[j] = __builtin_bit_cast(V, u);
  }
}

template <typename R, typename T, int VEC, int TEAM, int NV>
__global__ __launch_bounds__(TEAM ? 256 : 1024) void join_bwd_kernel(JoinArgs a, RowPlan pl) {
  constexpr int ROW = TEAM * NV * VEC;
  __shared__ float2 red[3][16];
  __shared__ float join[TEAM ? 256 * NV * VEC : 1];
  const JoinPlace p = join_place<TEAM>(pl);
  const RowPart<VEC, NV> rp(p.lane, TEAM ? TEAM : blockDim.x, a.C);
  const float inv_c = 1.0f / (float)a.C;
  const Act act = a.gate ? (Act)a.act : Act::kNone;
  const bool post = a.w_post != nullptr, pre = a.w_pre != nullptr;

  float wp[NV][VEC], sc[NV][VEC], wn[NV][VEC];
  load_weights<VEC, NV>(a.w_post, rp, 1.0f, wp);
  load_weights<VEC, NV>(a.scale, rp, 1.0f, sc);
  load_weights<VEC, NV>(a.w_pre, rp, 1.0f, wn);
  // Two vectors per lane: the weights live in LDS and are read where they are used (in registers they
  // would spill)
  __shared__ float lw[NV > 1 ? 3 * NV * VEC * 1024 : 1];
  if constexpr (NV > 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int at = ((j * VEC + i) * 3) * 1024 + threadIdx.x;
        lw[at] = wp[j][i];
        lw[at + 1024] = sc[j][i];
        lw[at + 2048] = wn[j][i];
      }
  }
  auto weight = [&](int k, int j, int i) {
    if constexpr (NV > 1) return lw[((j * VEC + i) * 3 + k) * 1024 + threadIdx.x];
    return k == 0 ? wp[j][i] : k == 1 ? sc[j][i] : wn[j][i];
  };
  float dwp[NV][VEC], dsc[NV][VEC], dwn[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) dwp[j][i] = dsc[j][i] = dwn[j][i] = 0.0f;
  const uint32_t team = (uint32_t)p.team, oo = team * (uint32_t)a.C;
  // A workgroup that is one team has its next row's loads on their way while it works on a row (few
  // such workgroups fit a CU); several teams in a workgroup hide each other's.
  constexpr bool AHEAD = TEAM == 0 && NV == 1;
  JoinBwdRow<R, T, VEC, NV> in, next;
  // Its stores have no branches around them: the wait for the next row's loads is then for those alone
  // (with a store that may not have been issued it is for every store too: 8192 rows of 4096 channels in
  // bf16 take 115 us, 123 with branches).
  auto put = [&](auto* base, int64_t t0, int j, const float(&v)[VEC], bool wanted = true) {
    using E = typename std::remove_pointer<decltype(base)>::type;
    if constexpr (AHEAD) {
      const auto row = buffer_rsrc(base + t0 * a.C, wanted ? (uint32_t)a.C * (uint32_t)sizeof(E) : 0u);
      buffer_store_vec<E, VEC>(row, row_offset<E, VEC, NV>(rp, j), v);
    } else if (wanted) {
      store_row<E, VEC, NV>(base + t0 * a.C, oo, rp, j, v);
    }
  };
  if (AHEAD && p.t0 < a.rows) next.load(a, p.t0, team, rp);
  for (int64_t t0 = p.t0; t0 < a.rows; t0 += p.step) {
    if (TEAM && t0 + p.team >= a.rows) break;
    if constexpr (AHEAD) {
      in = next;
      next.load(a, t0 + p.step < a.rows ? t0 + p.step : t0, team, rp);  // (the last row once more)
    } else {
      in.load(a, t0, team, rp);
    }
    if (!pre) {
#pragma unroll
      for (int j = 0; j < NV; ++j) in.dn[j] = (vec_t<T, VEC>)(T)0.0f;
    }
    float ry = 1.0f;
    if (post) {
      const float m =
          row_sum<VEC, NV>(rp, [&](int j, int i) { return (float)in.y[j][i] * (float)in.y[j][i]; });
      ry = rsqrtf(team_sum<TEAM>(m, red[0]) * inv_c + a.eps);
    }
    // r' and the two sums of its norm's backward
    if constexpr (NV > 1) renew(in.y);
    float ro[NV][VEC], av[NV][VEC], slope[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        av[j][i] = gate_act((float)in.g[j][i], act, slope[j][i]);
        const float yh = (float)in.y[j][i] * ry;
        ro[j][i] = fmaf(a.alpha * weight(1, j, i), yh * weight(0, j, i) * av[j][i], (float)in.r[j][i]);
      }
    float2 s;  // sum r'^2, sum dn w_pre r'
    s.x = row_sum<VEC, NV>(rp, [&](int j, int i) { return ro[j][i] * ro[j][i]; });
    s.y = row_sum<VEC, NV>(
        rp, [&](int j, int i) { return (float)in.dn[j][i] * weight(2, j, i) * ro[j][i]; });
    s = team_sum<TEAM>(s, red[1]);
    const float rr = pre ? rsqrtf(s.x * inv_c + a.eps) : 0.0f;
    const float c2 = rr * s.y * inv_c;
    if constexpr (NV > 1) {
      renew(in.y);
      renew(in.g);
      renew(in.dn);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float G[VEC], dg[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        if constexpr (NV > 1) av[j][i] = gate_act((float)in.g[j][i], act, slope[j][i]);
        const float rh = ro[j][i] * rr, d = (float)in.dn[j][i], yh = (float)in.y[j][i] * ry;
        const float y_act = yh * av[j][i], w = weight(0, j, i);
        G[i] = fmaf(rr, fmaf(-rh, c2, d * weight(2, j, i)), (float)in.dr[j][i]);
        const float du = a.alpha * weight(1, j, i) * G[i];
        dwn[j][i] = fmaf(d, rh, dwn[j][i]);
        dsc[j][i] = fmaf(G[i], y_act * w, dsc[j][i]);
        dwp[j][i] = fmaf(du, y_act, dwp[j][i]);
        const float duw = du * w;
        dg[i] = duw * yh * slope[j][i];
        ro[j][i] = duw * av[j][i];  // e from here on
      }
      put(static_cast<R*>(a.dres), t0, j, G);
      put(static_cast<T*>(a.dgate), t0, j, dg, a.gate != nullptr);
    }
    float c1 = 0.0f;
    if (post) {
      const float p1 = row_sum<VEC, NV>(
          rp, [&](int j, int i) { return ro[j][i] * ((float)in.y[j][i] * ry); });
      c1 = team_sum<TEAM>(p1, red[2]) * inv_c;
    }
    if constexpr (NV > 1) renew(in.y);
    // (with both of its sums a row's buffers are free again by the next one's)
    if (TEAM == 0 && !post) lds_barrier();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float dy[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) dy[i] = ry * fmaf(-((float)in.y[j][i] * ry), c1, ro[j][i]);
      put(static_cast<T*>(a.dy), t0, j, dy);
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (!(k == 0 ? a.w_post : k == 1 ? a.scale : a.w_pre)) continue;
    float* out = a.part + ((int64_t)blockIdx.x * 3 + k) * a.C;
    const float f = k == 1 ? a.alpha : 1.0f;
    if constexpr (TEAM != 0) lds_barrier();  // the readers of the weight before
    float* to = TEAM ? join + p.team * ROW : out;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (i >= rp.skip[j])
          to[rp.start[j] + i] = f * (k == 0 ? dwp[j][i] : k == 1 ? dsc[j][i] : dwn[j][i]);
    if constexpr (TEAM != 0) {
      lds_barrier();
      for (int c = threadIdx.x; c < a.C; c += 256) {
        float s = 0.0f;
#pragma unroll 4
        for (int q = 0; q < 256 / TEAM; ++q) s += join[q * ROW + c];
        out[c] = s;
      }
    }
  }
}

template <typename R, typename T, int VEC, bool BWD>
struct Launch {
  const RowPlan& pl;
  const JoinArgs& a;
  hipStream_t s;
  template <int TEAM, int NV>
  hipError_t run() const {
    const dim3 grid(pl.ntb), block(pl.nt);
    if constexpr (BWD)
      hipLaunchKernelGGL((join_bwd_kernel<R, T, VEC, TEAM, NV>), grid, block, 0, s, a, pl);
    else
      hipLaunchKernelGGL((join_kernel<R, T, VEC, TEAM, NV>), grid, block, 0, s, a, pl);
    return hipGetLastError();
  }
};
template <typename R, typename T, bool BWD>
static hipError_t launch_t(const RowPlan& pl, const JoinArgs& a, hipStream_t s) {
  constexpr Rows K = BWD ? Rows::kJoinBwd : Rows::kJoin;
  constexpr int W = wide_vec(K, sizeof(T));
  if (pl.vec > 1) return with_team<K, W>(pl, Launch<R, T, W, BWD>{pl, a, s});
  return with_team<K, 1>(pl, Launch<R, T, 1, BWD>{pl, a, s});
}
template <bool BWD>
static hipError_t launch_any(int dtype, int res_dtype, const RowPlan& pl, const JoinArgs& a,
                             hipStream_t s) {
  if (dtype == 1) return launch_t<float, float, BWD>(pl, a, s);
  return res_dtype == 1 ? launch_t<float, bf16, BWD>(pl, a, s) : launch_t<bf16, bf16, BWD>(pl, a, s);
}

hipError_t launch_join(int dtype, int res_dtype, const RowPlan& pl, const JoinArgs& a,
                       hipStream_t s) {
  return launch_any<false>(dtype, res_dtype, pl, a, s);
}
hipError_t launch_join_bwd(int dtype, int res_dtype, const RowPlan& pl, const JoinArgs& a,
                           hipStream_t s) {
  return launch_any<true>(dtype, res_dtype, pl, a, s);
}

}  // namespace gka
