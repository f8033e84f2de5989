// seq_delta_grad.hip -- the gradients of q, k, g and beta in each chunk of
// the gated delta rule, from the states around it, E and W = dL/dU (see
// seq_chunk.h and seq_delta_scan.hip).  With S the state before the chunk,
// dS the gradient of the state after it, dV = beta o W:
//   Ph = scale D o (dO U^T) (lower),  B = -D o (dV U^T) (strictly lower)
//   dQ = scale exp(G) o (dO S^T) + Ph K
//   dK = -exp(G) o (dV S^T) + exp(G_64 - G) o (U dS^T) + Ph^T Q + (B + B^T) K
//   dbeta_t = E_t . W_t
// g_s is in the exponent of every decay whose range holds it, so dg_s sums
// what each of these decays contributes:
//   exp(G_t), t >= s:             q_t . (scale exp(G) o (dO S^T))_t
//                                 - k_t . (exp(G) o (dV S^T))_t
//   exp(G_64 - G_j), j < s:       k_j . (exp(G_64 - G) o (U dS^T))_j
//   D_tj, j < s <= t:             Ph_tj (q_t . k_j) + B_tj (k_t . k_j)
//   exp(G_64):                    exp(G_64) <dS, S>
// Every term carries its own decay and none is the difference of larger
// ones: dg keeps its bits where it is small.  (q . dq - v . dv summed over
// the tokens from s on is the same number, but the pairs of a token with
// itself, which do not decay, are in both.)
//
// One workgroup of DP / 16 waves a (sequence, chunk, key head), the value
// heads that share the key head one after another, dv in blocks of 64
// columns.  A wave owns 16 key dimensions of dQ and dK, so the states go from
// memory to exactly one wave's registers; the operands that all waves share
// lie in LDS.
//
// Bound: waits (57% of the waves' time), at two waves a SIMD.  MI355X, 8x2048
// tokens of 16 heads, 128x128 states, bf16: 510 us; moving its 1.2 GB would
// take 250 us.  (With q . dq - v . dv for dg 446 us; that form with twice the
// waves 396 us, with registers spilled to memory, which no kernel here does.)
#include "../dwc_device.h"
#include "seq_chunk.h"

namespace dwc {
namespace seq {
namespace grad {

constexpr int kPitch = 72;             // halves a row: 144 bytes, 16-byte aligned
constexpr int kTile = kChunk * kPitch;  // halves a 64x64 tile

// 8 consecutive halves at column 32 ks + 8 q.
__device__ __forceinline__ half8 frag8(const _Float16* tile, int row, int ks, int q) {
  return *(const half8*)(tile + row * kPitch + 32 * ks + 8 * q);
}

// 8 halves in the order of the packed K and Q fragments.
__device__ __forceinline__ half8 frag44(const _Float16* tile, int row, int ks, int q) {
  const half4 u = *(const half4*)(tile + row * kPitch + 32 * ks + 4 * q);
  const half4 v = *(const half4*)(tile + row * kPitch + 32 * ks + 16 + 4 * q);
  return half8{u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
}

// Pieces of N consecutive values to a row of a tile.
template <int P, int N>
__device__ __forceinline__ void put(_Float16* tile, int row, int col, const float* v, float s) {
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    half8 hi, lo;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      _Float16 h, l;
      split(v[i + j] * s, &h, &l);
      hi[j] = h;
      lo[j] = l;
    }
    *(half8*)(tile + row * kPitch + col + i) = hi;
    if constexpr (P == 2) *(half8*)(tile + kTile + row * kPitch + col + i) = lo;
  }
}

// LDS tiles: dO, dV, U per block of dv, then Ph, Ph^T, B + B^T, two pieces
// each.
constexpr int kLds = 6 * kTile * 2;

template <int V>
struct Int {
  static constexpr int value = V;
};

// Waves a SIMD that leave a wave registers for all it holds.
constexpr int waves_of(int dp, bool shared) { return dp == 64 && shared ? 1 : 2; }

// SHARED: value heads share a key head, whose gradients are their sums.
template <int T, int DP, bool SHARED>
__global__ void __launch_bounds__(DP * 4, waves_of(DP, SHARED)) delta_grad(ChunkArgs c) {
  constexpr int NP = T == T_F32 ? 2 : 1;  // pieces of an input
  constexpr int NW = DP / 16;   // waves
  constexpr int CPT = 64 / NW;  // columns of a 64-wide tile a thread loads
  extern __shared__ __align__(16) char lds_raw[];
  __shared__ float red[3][NW];
  // each wave's part of what the decays exp(G_t), exp(G_64 - G_j) and D take
  // to dg
  __shared__ float sinto_g[NW][kChunk], sout_g[NW][kChunk], spair_g[NW][kChunk], sbeta[kChunk];
  __shared__ __align__(16) float sinto[kChunk], sout[kChunk];
  __shared__ double sg[kChunk];
  _Float16* lds = (_Float16*)lds_raw;
  _Float16 *tdo = lds, *tdv = lds + 2 * kTile, *tu = lds + 4 * kTile;
  _Float16 *tph = lds, *tpt = lds + 2 * kTile, *tb = lds + 4 * kTile;
  const DeltaArgs& a = c.a;
  const int tid = threadIdx.x, lane = tid & 63, m0 = lane & 15, q0 = lane >> 4;
  const int w = uniform(tid >> 6);
  const int row0 = tid / NW, part0 = tid % NW;  // for whole-tile loads
  const int64_t id = blockIdx.x;
  const int hk = (int)(id % a.hk);
  const int64_t bc = id / a.hk;
  const int chunk = (int)(bc % c.nc);
  const int64_t b = bc / c.nc;
  const int64_t len = live_tokens(a, b), t0 = (int64_t)chunk * kChunk;
  const int n = (int)(len - t0 < 0 ? 0 : (len - t0 < kChunk ? len - t0 : kChunk));
  const int per = SHARED ? a.hv / a.hk : 1;
  f32x4 dq[4], dk[4], dqs[4];  // dqs: of the heads before this one
#pragma unroll
  for (int i = 0; i < 4; ++i) dq[i] = dk[i] = dqs[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  // this wave's key dimension: 16 w + lane % 16
  const Frag* kt = c.kt + (id * NP * (DP / 16 * 2) + w * 2) * 64;
  const Frag* qt = c.qt + (id * NP * (DP / 16 * 2) + w * 2) * 64;
  const uint32_t loff = 16 * lane;
  constexpr int PIECE = DP / 16 * 2 * 64;

  for (int r = 0; r < per; ++r) {
    const int h = hk * per + r;
    const int64_t hid = bc * a.hv + h;
    // opaque copies, so that addresses made of them are made again for each
    // head instead of held through the loop (they would not fit)
    int m = m0, q = q0, row = row0, part = part0;
    asm volatile("" : "+v"(m), "+v"(q), "+v"(row), "+v"(part));
    if (n == 0) {  // past the sequence: zeros
      if (tid < kChunk && t0 + tid < a.l) {
        a.dg[(b * a.l + t0 + tid) * a.hv + h] = 0.f;
        a.dbeta[(b * a.l + t0 + tid) * a.hv + h] = 0.f;
      }
      continue;
    }
    const Gate* gate = c.gate + hid;
    const float beta = gate->beta[row], kinv = gate->kinv, qinv = gate->qinv;
    float ew = 0.f, sds = 0.f;
    // this wave's key dimensions of k . dk by the decays exp(G) and exp(G_64 - G)
    f32x4 kin[4], kout[4];
    // rows 16 wr.., columns 16 j.. of dO U^T and dV U^T: with 8 waves four
    // of them take the one and four the other, with 4 waves each takes both
    constexpr int BOTH = NW == 4 ? 2 : 1;
    const int wr = w & 3;
    f32x4 dp[BOTH][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      kin[i] = kout[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int x = 0; x < BOTH; ++x) dp[x][i] = f32x4{0.f, 0.f, 0.f, 0.f};
      if constexpr (SHARED) {
        dqs[i] += dq[i];
        dq[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
    }
    for (int v0 = 0; v0 < c.dvp; v0 += 64) {
      __syncthreads();  // the tiles' readers are done
      if (v0 == 0 && tid < kChunk) {
        sg[tid] = gate->g[tid];
        sinto[tid] = gate->into[tid];
        sout[tid] = gate->out[tid];
      }
      asm volatile("" : "+v"(m), "+v"(q), "+v"(row), "+v"(part));
      float xd[CPT], xv[CPT], xu[CPT];
      float md = 0.f, mv = 0.f, mu = 0.f;
      {
        const int col = v0 + CPT * part;
        const int64_t t = t0 + row;
        const float* ep = c.e + (hid * kChunk + row) * c.dvp + col;
        const float* wp = c.dw + (hid * kChunk + row) * c.dvp + col;
        const int64_t ob = b * a.do_stride[0] + t * a.do_stride[1] + h * a.do_stride[2] + col;
#pragma unroll
        for (int i = 0; i < CPT; ++i) xd[i] = xv[i] = xu[i] = 0.f;
        if (c.wide) {  // dv is a multiple of 8: eight columns are in or out
#pragma unroll
          for (int i = 0; i < CPT; i += 8)
            if (row < n && col + i < a.dv) load_vec<T, 8>(a.dout, ob + i, xd + i);
        } else {
#pragma unroll
          for (int i = 0; i < CPT; ++i)
            if (row < n && col + i < a.dv) xd[i] = load1<T>(a.dout, ob + i);
        }
        if (col < c.dvp) {
          load_vec<T_F32, CPT>(ep, 0, xu);
          load_vec<T_F32, CPT>(wp, 0, xv);
        }
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          ew = fmaf(xu[i], xv[i], ew);
          xv[i] *= beta;
          xu[i] *= beta;
          md = fmaxf(md, fabsf(xd[i]));
          mv = fmaxf(mv, fabsf(xv[i]));
          mu = fmaxf(mu, fabsf(xu[i]));
        }
      }
      md = wave_max(md);
      mv = wave_max(mv);
      mu = wave_max(mu);
      if (lane == 0) {
        red[0][w] = md;
        red[1][w] = mv;
        red[2][w] = mu;
      }
      __syncthreads();
      md = mv = mu = 0.f;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        md = fmaxf(md, red[0][i]);
        mv = fmaxf(mv, red[1][i]);
        mu = fmaxf(mu, red[2][i]);
      }
      const Scale sd = scale_of(md), sv = scale_of(mv), su = scale_of(mu);
      put<NP, CPT>(tdo, row, CPT * part, xd, sd.mul);
      put<2, CPT>(tdv, row, CPT * part, xv, sv.mul);
      put<2, CPT>(tu, row, CPT * part, xu, su.mul);
      __syncthreads();
      // dO U^T and dV U^T
      const auto lower = [&](auto pieces, const _Float16* tile, float inv, f32x4(&acc)[4]) {
        constexpr int P = decltype(pieces)::value;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j > wr) break;
          __builtin_amdgcn_sched_barrier(0);
          f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            half8 f[P], fu[2];
#pragma unroll
            for (int y = 0; y < P; ++y) f[y] = frag8(tile + y * kTile, 16 * wr + m, ks, q);
#pragma unroll
            for (int y = 0; y < 2; ++y) fu[y] = frag8(tu + y * kTile, 16 * j + m, ks, q);
            p = mfma_pieces<P, 2>(f, fu, p);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[j][i] = fmaf(inv, p[i], acc[j][i]);
        }
      };
      if (BOTH == 2 || w < 4) lower(Int<NP>{}, tdo, sd.inv * su.inv, dp[0]);
      if (BOTH == 2 || w >= 4) lower(Int<2>{}, tdv, sv.inv * su.inv, dp[BOTH - 1]);
      // dO S^T, dV S^T and U dS^T
      asm volatile("" : "+v"(m), "+v"(q), "+v"(row), "+v"(part));
      {
        const int64_t at = (hid * DP + 16 * w + m) * c.dvp + v0 + 8 * q;
        f32x4 s[4], g[4];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const bool in = v0 + 32 * ks + 8 * q < c.dvp;
            s[2 * ks + x] = in ? *(const f32x4*)(c.states + at + 32 * ks + 4 * x)
                               : f32x4{0.f, 0.f, 0.f, 0.f};
            g[2 * ks + x] = in ? *(const f32x4*)(c.dstates + at + 32 * ks + 4 * x)
                               : f32x4{0.f, 0.f, 0.f, 0.f};
          }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int x = 0; x < 4; ++x) sds = fmaf(s[i][x], g[i][x], sds);
        half8 fk[2][NP];
        const auto load_k = [&]() {
          uint32_t at = loff;
          asm volatile("" : "+v"(at));  // loaded again, not held, where it says so
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int y = 0; y < NP; ++y) fk[ks][y] = at_lane(kt + y * PIECE + ks * 64, at);
        };
        load_k();
        // k at the place of value x of row block i of a result, from its
        // fragments
        const auto k_at = [&](int i, int x) {
          const int slot = (i & 1) * 4 + x;
          float v = (float)fk[i >> 1][0][slot];
          if constexpr (NP == 2) v += (float)fk[i >> 1][1][slot];
          return v;
        };
        // one state after the other: fragments of both would not fit
        {
          const Scale ss = scale_of(column_max(abs_max(s)));
          half8 fs[2][2];
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) to_frag<2>(s[2 * ks], s[2 * ks + 1], ss.mul, fs[ks]);
          const float cq = a.scale * sd.inv, ck = -sv.inv;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // loads of later rows are not pulled ahead of this one's products
            __builtin_amdgcn_sched_barrier(0);
            f32x4 xq = {0.f, 0.f, 0.f, 0.f}, xk = xq;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
              half8 fo[NP];
#pragma unroll
              for (int y = 0; y < NP; ++y) fo[y] = frag8(tdo + y * kTile, 16 * i + m, ks, q);
              const half8 fv[2] = {frag8(tdv, 16 * i + m, ks, q),
                                   frag8(tdv + kTile, 16 * i + m, ks, q)};
              xq = mfma_pieces<NP, 2>(fo, fs[ks], xq);
              xk = mfma_pieces<2, 2>(fv, fs[ks], xk);
            }
            const f32x4 into = *(const f32x4*)(sinto + 16 * i + 4 * q);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              dq[i][x] = fmaf(cq * into[x], ss.inv * xq[x], dq[i][x]);
              const float v = ck * into[x] * (ss.inv * xk[x]);
              kin[i][x] = fmaf(k_at(i, x), v, kin[i][x]);
              dk[i][x] += v;
            }
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        {
          const Scale sgr = scale_of(column_max(abs_max(g)));
          half8 fg[2][2];
          if constexpr (SHARED && NP == 2) load_k();  // (no registers to hold it)
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) to_frag<2>(g[2 * ks], g[2 * ks + 1], sgr.mul, fg[ks]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            f32x4 xs = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
              const half8 fu[2] = {frag8(tu, 16 * i + m, ks, q),
                                   frag8(tu + kTile, 16 * i + m, ks, q)};
              xs = mfma_pieces<2, 2>(fu, fg[ks], xs);
            }
            const f32x4 out = *(const f32x4*)(sout + 16 * i + 4 * q);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float v = su.inv * out[x] * (sgr.inv * xs[x]);
              kout[i][x] = fmaf(k_at(i, x), v, kout[i][x]);
              dk[i][x] += v;
            }
          }
        }
      }
    }
    // Ph, Ph^T and B + B^T to LDS
    asm volatile("" : "+v"(m), "+v"(q), "+v"(row), "+v"(part));
    __syncthreads();
    float mx[2] = {0.f, 0.f};
    f32x4 pair[4];  // what the decay of each pair of tokens contributes
#pragma unroll
    for (int j = 0; j < 4; ++j) pair[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < BOTH; ++x) {
      const bool ph = BOTH == 2 ? x == 0 : w < 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j > wr) continue;  // zero as it is
        const f32x4 with =
            (ph ? c.qk : c.kk)[(id * kLow + low_block(wr, j)) * 64 + 16 * q + m];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = 16 * wr + 4 * q + i, cc = 16 * j + m;
          const float d = cc <= rr ? __builtin_amdgcn_exp2f((float)(sg[rr] - sg[cc])) : 0.f;
          const float v = ph ? a.scale * d * dp[x][j][i] : -d * dp[x][j][i];
          if (cc < rr) pair[j][i] = fmaf(v, with[i], pair[j][i]);
          dp[x][j][i] = cc < rr || (ph && cc == rr) ? v : 0.f;
          mx[x] = fmaxf(mx[x], fabsf(dp[x][j][i]));
        }
      }
    }
    // The pairs (t, j) with j < s <= t, summed for each s: over j < s inside
    // each row t, then over this wave's rows t >= s.
    {
      f32x4 before = {0.f, 0.f, 0.f, 0.f};  // of the blocks left of this one
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float sum = 0.f;
        if (j <= wr) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (16 * j + m <= 16 * wr + 4 * q + i) sum += before[i] + sum_before16(pair[j][i]);
            before[i] += lane_sum<16>(pair[j][i]);
          }
          float o;
          rows16(sum, o);
          sum += o;
          halves(sum, o);
          sum += o;
        }
        if (q == 0) spair_g[w][16 * j + m] = sum;
      }
    }
    if (BOTH == 1 && w >= 4) {
      mx[1] = mx[0];
      mx[0] = 0.f;
    }
    mx[0] = wave_max(mx[0]);
    mx[1] = wave_max(mx[1]);
    if (lane == 0) {
      red[0][w] = mx[0];
      red[1][w] = mx[1];
    }
    __syncthreads();
    mx[0] = mx[1] = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      mx[0] = fmaxf(mx[0], red[0][i]);
      mx[1] = fmaxf(mx[1], red[1][i]);
    }
    const Scale sp = scale_of(mx[0]), sb = scale_of(mx[1]);
#pragma unroll
    for (int y = 0; y < BOTH; ++y) {
      const bool ph = BOTH == 2 ? y == 0 : w < 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // four rows of a column: together in the transposes
        half4 hi, lo;
        const int r4 = 16 * wr + 4 * q, cc = 16 * j + m;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          _Float16 h, l;
          split(dp[y][j][i] * (ph ? sp.mul : sb.mul), &h, &l);
          hi[i] = h;
          lo[i] = l;
        }
        if (ph) {
          *(half4*)(tpt + cc * kPitch + r4) = hi;
          *(half4*)(tpt + kTile + cc * kPitch + r4) = lo;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            tph[(r4 + i) * kPitch + cc] = hi[i];
            tph[kTile + (r4 + i) * kPitch + cc] = lo[i];
          }
        } else if (j < wr) {
          *(half4*)(tb + cc * kPitch + r4) = hi;
          *(half4*)(tb + kTile + cc * kPitch + r4) = lo;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            tb[(r4 + i) * kPitch + cc] = hi[i];
            tb[kTile + (r4 + i) * kPitch + cc] = lo[i];
          }
        } else if (j == wr) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (cc > r4 + i) continue;
            tb[(r4 + i) * kPitch + cc] = hi[i];
            tb[cc * kPitch + r4 + i] = hi[i];
            tb[kTile + (r4 + i) * kPitch + cc] = lo[i];
            tb[kTile + cc * kPitch + r4 + i] = lo[i];
          }
        }
      }
    }
    __syncthreads();
    asm volatile("" : "+v"(m), "+v"(q), "+v"(row), "+v"(part));
    {
      half8 fq[2][NP], fk[2][NP];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int y = 0; y < NP; ++y) {
          fq[ks][y] = at_lane(qt + y * PIECE + ks * 64, loff);
          fk[ks][y] = at_lane(kt + y * PIECE + ks * 64, loff);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        f32x4 xq = {0.f, 0.f, 0.f, 0.f}, xp = xq, xb = xq;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          if (ks == 0 || i >= 2) {
            const half8 f[2] = {frag44(tph, 16 * i + m, ks, q),
                                frag44(tph + kTile, 16 * i + m, ks, q)};
            xq = mfma_pieces<2, NP>(f, fk[ks], xq);
          }
          half8 f[2], g[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            f[y] = frag44(tpt + y * kTile, 16 * i + m, ks, q);
            g[y] = frag44(tb + y * kTile, 16 * i + m, ks, q);
          }
          if (ks == 1 || i < 2) xp = mfma_pieces<2, NP>(f, fq[ks], xp);
          xb = mfma_pieces<2, NP>(g, fk[ks], xb);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          // q at this place, from its fragments; dq is by exp(G) so far
          const int slot = (i & 1) * 4 + x;
          float qv = (float)fq[i >> 1][0][slot];
          if constexpr (NP == 2) qv += (float)fq[i >> 1][1][slot];
          const float in = lane_sum<16>(fmaf(qv * qinv, dq[i][x], kinv * kin[i][x]));
          const float out = lane_sum<16>(kinv * kout[i][x]);
          if (m == 0) {
            sinto_g[w][16 * i + 4 * q + x] = in;
            sout_g[w][16 * i + 4 * q + x] = out;
          }
          dq[i][x] = fmaf(sp.inv * kinv, xq[x], dq[i][x]);
          dk[i][x] += fmaf(sp.inv * qinv, xp[x], sb.inv * kinv * xb[x]);
        }
      }
    }
    // dbeta and dg
    ew = lane_sum<NW>(ew);
    if (part == 0) sbeta[row] = ew;
    sds = lane_sum<64>(sds);
    if (lane == 0) red[2][w] = sds;
    __syncthreads();
    if (w == 0) {
      float d = 0.f, early = 0.f, pairs = 0.f, far = 0.f;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        d += sinto_g[i][lane];
        if (lane > 0) early += sout_g[i][lane - 1];
        pairs += spair_g[i][lane];
        far += red[2][i];
      }
      // over the tokens from this one on, and over those before it
#pragma unroll
      for (int i = 1; i < 64; i <<= 1) {
        const float o = __shfl_down(d, i, 64), p = __shfl_up(early, i, 64);
        if (lane + i < 64) d += o;
        if (lane >= i) early += p;
      }
      d += early + pairs + gate->total * far;
      if (t0 + lane < a.l) {
        a.dg[(b * a.l + t0 + lane) * a.hv + h] = lane < n ? d : 0.f;
        a.dbeta[(b * a.l + t0 + lane) * a.hv + h] = lane < n ? sbeta[lane] : 0.f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int t = 16 * i + 4 * q0 + x, col = 16 * w + m0;
        if (t0 + t >= a.l || col >= a.dk) continue;
        const int64_t at = ((b * a.l + t0 + t) * a.hk + hk) * a.dk + col;
        store1<T>(a.dq, at, t < n ? dqs[i][x] + dq[i][x] : 0.f);
        store1<T>(a.dk_out, at, t < n ? dk[i][x] : 0.f);
      }
}

template <int T>
void go(const ChunkArgs& c, hipStream_t st) {
  const dim3 grid((uint32_t)(c.a.b * c.nc * c.a.hk));
  if (c.a.hv == c.a.hk) {
    if (c.a.dk <= 64) hipLaunchKernelGGL((delta_grad<T, 64, false>), grid, dim3(256), kLds, st, c);
    else hipLaunchKernelGGL((delta_grad<T, 128, false>), grid, dim3(512), kLds, st, c);
  } else {
    if (c.a.dk <= 64) hipLaunchKernelGGL((delta_grad<T, 64, true>), grid, dim3(256), kLds, st, c);
    else hipLaunchKernelGGL((delta_grad<T, 128, true>), grid, dim3(512), kLds, st, c);
  }
}

}  // namespace grad

hipError_t launch_delta_grad(ChunkArgs c, hipStream_t st) {
  const int64_t unit = c.a.type == T_F32 ? 4 : 8;
  c.wide = c.a.dv % 8 == 0 && (uintptr_t)c.a.dout % 16 == 0;
  for (int i = 0; i < 3; ++i) c.wide = c.wide && c.a.do_stride[i] % unit == 0;
  if (c.a.type == T_F32) grad::go<T_F32>(c, st);
  else if (c.a.type == T_BF16) grad::go<T_BF16>(c, st);
  else grad::go<T_F16>(c, st);
  return hipGetLastError();
}

}  // namespace seq
}  // namespace dwc
