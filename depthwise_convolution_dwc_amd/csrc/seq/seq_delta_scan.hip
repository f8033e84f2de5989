// seq_delta_scan.hip -- the serial part of the chunked gated delta rule, and
// of its gradient (formulas in seq_chunk.h).
//
// A column of the state depends on no other, so a workgroup owns 16 NT
// columns of one head for the whole sequence.  Its two waves share them by
// rows: each holds half of the state (fp32, as 16x16 results of the matrix
// cores) and makes the results of half of a chunk's tokens.  Every product
// has the state, or something made of it, on the right; its rows are 32-row
// blocks that one wave owns whole, so a block's scale needs no other wave,
// and the blocks go through LDS (three exchanges a chunk).  The fragments on
// the left are each wave's own: they go from memory to registers, each
// refilled for the next chunk once this chunk is done with it, so that no
// exchange waits for memory.  (Issued before an exchange they hold up the
// wave's partner, after it the products that follow: forward the former is
// faster, 194 against 207 us at 8x2048 tokens of 16 heads with one fp16
// number an operand of o; beside the stores of the backward scans the latter,
// 455 against 505 us.)
//
// Bound: the chain of products and exchanges of a chunk (a wave issues half
// of its cycles, three quarters of that vector instructions; the matrix
// cores are busy 16% of the time), times the chunks of the longest sequence.
// MI355X, 128x128 states, bf16: 2.8 us a chunk at one workgroup a compute unit
// (4096 tokens of 32 heads: 181 us), 6.8 us where every SIMD has a wave with
// 32 columns (8x2048 tokens of 16 heads: 217 us).
#include "../dwc_device.h"
#include "seq_chunk.h"

namespace dwc {
namespace seq {
namespace scans {

// The 4 fp32 values of rows 16 i + 4 q .. + 3.
__device__ __forceinline__ f32x4 row4(const float* p, int i, int q) {
  return *(const f32x4*)(p + 16 * i + 4 * q);
}

// LDS written before is visible to both waves after; loads from memory stay
// in flight (__syncthreads may wait for them).
__device__ __forceinline__ void exchange() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

template <int T>
struct Raw {
  typedef uint16_t type;
  static __device__ __forceinline__ float value(uint16_t x) { return from16<T>(x); }
};
template <>
struct Raw<T_F32> {
  typedef float type;
  static __device__ __forceinline__ float value(float x) { return x; }
};

// This wave's rows of a chunk's gates.
struct Gates {
  f32x4 into[2], out[2], beta[2];
  float total, xinv, pinv, kinv, qinv, top, kpart, qpart;
  __device__ __forceinline__ void load(const Gate* g, int hf, int q) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      into[x] = row4(g->into, 2 * hf + x, q);
      out[x] = row4(g->out, 2 * hf + x, q);
      beta[x] = row4(g->beta, 2 * hf + x, q);
    }
    total = g->total;
    xinv = g->xinv;
    pinv = g->pinv;
    kinv = g->kinv;
    qinv = g->qinv;
    top = g->top;
    kpart = g->kpart;
    qpart = g->qpart;
  }
};

// A block of 32 rows of an operand in LDS: both pieces, and what its columns'
// values are to be multiplied by.
struct Block {
  half8 f[2][64];
  float inv[16];
};

template <int P>
__device__ __forceinline__ void publish(Block* blk, const f32x4& t0, const f32x4& t1,
                                        const Scale& s, int lane) {
  half8 f[2];
  to_frag<P>(t0, t1, s.mul, f);
  blk->f[0][lane] = f[0];
  if constexpr (P == 2) blk->f[1][lane] = f[1];
  if (lane < 16) blk->inv[lane] = s.inv;
}

__device__ __forceinline__ float abs_max2(const f32x4 (&v)[2]) { return abs_max(v); }

// The blocks of two waves that share columns.
template <int KS, int NT, bool BWD>
struct Blocks {
  Block bs[NT][KS], by[NT][2], bu[NT][2], bo[BWD ? 1 : NT][2];
};
template <int KS, int NT>
struct BlocksBack {
  Block bs[NT][KS], by[NT][2], bu[NT][2], bo[NT][2], bd[NT][2];
};

// What both kernels know of their place.
struct Place {
  int64_t b, head;
  int h, hk, block, col0;  // block: the first column, col0: this lane's
};

template <int NT, int NC>
__device__ __forceinline__ Place place_of(const ChunkArgs& c, int block, int blocks) {
  Place p;
  const DeltaArgs& a = c.a;
  const int groups = (c.dvp / 16 + NT * NC - 1) / (NT * NC);
  // the workgroups of one head read the same fragments: on one XCD's L2
  const int id = xcd_logical_block(block, blocks);
  p.head = id / groups;
  // (past dvp for the last pair of waves of an odd number of blocks, which
  // then only keeps the exchanges company)
  p.block = ((int)(id - p.head * groups) * NC + uniform((int)threadIdx.x >> 7)) * 16 * NT;
  p.col0 = p.block + (threadIdx.x & 15);
  p.b = p.head / a.hv;
  p.h = (int)(p.head - p.b * a.hv);
  p.hk = p.h / (a.hv / a.hk);
  return p;
}

// This wave's 32 rows of a chunk in a tensor of tokens.
template <int T, int NT>
struct Rows {
  char* lane;      // token 4 q of this wave's rows in the first chunk, column col0
  int64_t stride;  // bytes between tokens
  __device__ __forceinline__ Rows(const void* t, const int64_t (&st)[3], const Place& p, int hf,
                                  int q)
      : stride(st[1] * E) {
    lane = (char*)t + (p.b * st[0] + p.h * st[2] + p.col0) * E + (32 * hf + 4 * q) * stride;
  }
  // a dense output
  __device__ __forceinline__ Rows(void* t, int64_t l, int hv, int dv, const Place& p, int hf,
                                  int q)
      : stride((int64_t)hv * dv * E) {
    lane = (char*)t + ((p.b * l * hv + p.h) * dv + p.col0) * E + (32 * hf + 4 * q) * stride;
  }
  // A chunk inside the sequence needs no look at each token.
  __device__ __forceinline__ void load(typename Raw<T>::type (&f)[NT][2][4], int chunk,
                                       int64_t len, bool whole, const bool (&ok)[NT], int hf,
                                       int q) const {
    const int64_t t0 = (int64_t)chunk * kChunk;
    const char* at = lane + t0 * stride;
    if (whole && t0 + kChunk <= len) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            f[nt][x][r] = ((const typename Raw<T>::type*)(at + (16 * x + r) * stride))[16 * nt];
    } else {
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            f[nt][x][r] = 0;
            if (ok[nt] && t0 + 32 * hf + 16 * x + 4 * q + r < len)
              f[nt][x][r] = ((const typename Raw<T>::type*)(at + (16 * x + r) * stride))[16 * nt];
          }
    }
  }
  // Rows past the sequence's length are written as zeros.
  __device__ __forceinline__ void store(const f32x4 (&f)[NT][2], int chunk, int64_t len, int64_t l,
                                        bool whole, const bool (&ok)[NT], int hf, int q) const {
    const int64_t t0 = (int64_t)chunk * kChunk;
    char* at = lane + t0 * stride;
    if (whole && t0 + kChunk <= len) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            store1<T>(at + (16 * x + r) * stride, 16 * nt, f[nt][x][r]);
    } else {
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int64_t t = t0 + 32 * hf + 16 * x + 4 * q + r;
            if (ok[nt] && t < l)
              store1<T>(at + (16 * x + r) * stride, 16 * nt, t < len ? f[nt][x][r] : 0.f);
          }
    }
  }

 private:
  static constexpr int64_t E = ElemBytes<T>::value;
};

// Values of a 16-row result to rows row0 + 4 q + r of a matrix of dvp
// columns, the matrix at a uniform address.
__device__ __forceinline__ void store_tile(float* matrix, int row0, int dvp, uint32_t offset,
                                           const f32x4& v) {
#pragma unroll
  for (int r = 0; r < 4; ++r)
    *(float*)((char*)(matrix + (int64_t)(row0 + r) * dvp) + offset) = v[r];
}

// NT: 16-column blocks of a wave.  NC: pairs of waves of a workgroup.
// block of blocks: the workgroup's number among those of its kind.
template <int T, int DP, int NT, int NC, bool BWD>
__device__ __forceinline__ void scan(const ChunkArgs& c, int block, int blocks, char* lds) {
  constexpr int NP = T == T_F32 ? 2 : 1;
  constexpr int KS = DP / 32, MT = DP / 16, MW = MT / 2;
  typedef Raw<T> R;
  auto& [bs, by, bu, bo] = ((Blocks<KS, NT, BWD>*)lds)[uniform((int)threadIdx.x >> 7)];
  const DeltaArgs& a = c.a;
  const Place p = place_of<NT, NC>(c, block, blocks);
  const int lane = threadIdx.x & 63, hf = uniform((int)threadIdx.x >> 6) & 1;
  const int m = lane & 15, q = lane >> 4;
  const int64_t len = live_tokens(a, p.b);
  const int chunks = (int)((len + kChunk - 1) / kChunk);
  const uint32_t loff = 16 * lane, soff = 4 * (4 * q * c.dvp + p.col0);
  const bool whole = p.block + 16 * NT <= a.dv;  // no column past the head size
  bool ok[NT], in[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    ok[nt] = p.col0 + 16 * nt < a.dv;
    in[nt] = p.block + 16 * nt < c.dvp;
  }

  f32x4 s[NT][MW];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < MW; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * (hf * MW + i) + 4 * q + r;
        s[nt][i][r] = a.s0 && ok[nt] && row < a.dk
                          ? a.s0[(p.head * a.dk + row) * a.dv + p.col0 + 16 * nt] : 0.f;
      }

  // this wave's fragments and values of one chunk
  half8 ka[2][KS][NP], kt[MW][2][NP], xa[2][2][2], qa[2][KS][NP], pa[2][2][2];
  typename R::type vr[NT][2][4];
  Gates gt, gn;
  const auto kid_of = [&](int chunk) { return (p.b * c.nc + chunk) * a.hk + p.hk; };
  const auto hid_of = [&](int chunk) { return (p.b * c.nc + chunk) * a.hv + p.h; };
  const auto load_rows = [&](half8(&f)[2][KS][NP], const Frag* base, int chunk) {
    const Frag* src = base + kid_of(chunk) * NP * 4 * KS * 64;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int y = 0; y < NP; ++y) f[x][ks][y] = at_lane(src + ((y * 4 + 2 * hf + x) * KS + ks) * 64, loff);
  };
  const auto load_kt = [&](int chunk) {
    const Frag* src = c.kt + kid_of(chunk) * NP * MT * 2 * 64;
#pragma unroll
    for (int i = 0; i < MW; ++i)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int y = 0; y < NP; ++y)
          kt[i][ks][y] = at_lane(src + ((y * MT + hf * MW + i) * 2 + ks) * 64, loff);
  };
  // rows 0..31 of a lower triangular operand have their first block only
  const auto load_tri = [&](half8(&f)[2][2][2], const Frag* base, int chunk) {
    const Frag* src = base + hid_of(chunk) * 2 * kTri * 64;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int y = 0; y < 2; ++y)
          if (ks == 0 || hf)
            f[x][ks][y] = at_lane(src + (y * kTri + (hf ? 2 + 2 * x + ks : x)) * 64, loff);
  };
  const Rows<T, NT> rows_v(a.v, a.v_stride, p, hf, q), rows_o(a.o, a.l, a.hv, a.dv, p, hf, q);
  const auto load_v = [&](int chunk) { rows_v.load(vr, chunk, len, whole, ok, hf, q); };
  if (chunks > 0) {
    gt.load(c.gate + hid_of(0), hf, q);
    load_rows(ka, c.ka, 0);
    load_v(0);
    if constexpr (!BWD) load_rows(qa, c.qa, 0);
    load_tri(xa, c.xa, 0);
    load_kt(0);
    if constexpr (!BWD) load_tri(pa, c.pa, 0);
  }
  for (int chunk = 0; chunk < chunks; ++chunk) {
    const int next = chunk + 1 < chunks ? chunk + 1 : chunk;
    const int64_t hid = hid_of(chunk);
    gn.load(c.gate + hid_of(next), hf, q);
    // the state's blocks of this wave
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const Scale ss = scale_of(column_max(abs_max(s[nt])));
#pragma unroll
      for (int i = 0; i < MW; i += 2)
        publish<2>(&bs[nt][(hf * MW + i) / 2], s[nt][i], s[nt][i + 1], ss, lane);
    }
    exchange();
    // e = V - exp(G) o (K S)
    f32x4 e[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      f32x4 acc[2][2] = {};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const half8 f[2] = {bs[nt][ks].f[0][lane], bs[nt][ks].f[1][lane]};
#pragma unroll
        for (int x = 0; x < 2; ++x)
          acc[x][ks / (KS / 2)] = mfma_pieces<NP, 2>(ka[x][ks], f, acc[x][ks / (KS / 2)]);
      }
      const float i0 = gt.kinv * bs[nt][0].inv[m], i1 = gt.kinv * bs[nt][KS - 1].inv[m];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          e[nt][x][r] = R::value(vr[nt][x][r]) -
                        gt.into[x][r] * fmaf(i0, acc[x][0][r], i1 * acc[x][1][r]);
    }
    load_rows(ka, c.ka, next);
    load_v(next);
    f32x4 u[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int x = 0; x < 2; ++x) u[nt][x] = gt.beta[x] * e[nt][x];
      publish<2>(&by[nt][hf], u[nt][0], u[nt][1], scale_of(column_max(abs_max2(u[nt]))), lane);
    }
    // Q S, while the other wave's block is on its way
    f32x4 o[NT][2];
    if constexpr (!BWD) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        f32x4 acc[2][2] = {};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const half8 f[2] = {bs[nt][ks].f[0][lane], bs[nt][ks].f[1][lane]};
#pragma unroll
          for (int x = 0; x < 2; ++x)
            acc[x][ks / (KS / 2)] = mfma_pieces<NP, 2>(qa[x][ks], f, acc[x][ks / (KS / 2)]);
        }
        const float sc = a.scale * gt.qinv;
        const float i0 = sc * bs[nt][0].inv[m], i1 = sc * bs[nt][KS - 1].inv[m];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            o[nt][x][r] = gt.into[x][r] * fmaf(i0, acc[x][0][r], i1 * acc[x][1][r]);
      }
      load_rows(qa, c.qa, next);
    }
    exchange();
    // E = e - X (beta o e), U = beta o E
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      f32x4 acc[2][2] = {};
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (ks > hf) break;
        const half8 f[2] = {by[nt][ks].f[0][lane], by[nt][ks].f[1][lane]};
#pragma unroll
        for (int x = 0; x < 2; ++x) acc[x][ks] = mfma_pieces<2, 2>(xa[x][ks], f, acc[x][ks]);
      }
      const float i0 = gt.xinv * by[nt][0].inv[m], i1 = gt.xinv * by[nt][1].inv[m];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int r = 0; r < 4; ++r) e[nt][x][r] -= fmaf(i0, acc[x][0][r], i1 * acc[x][1][r]);
        u[nt][x] = gt.beta[x] * e[nt][x];
      }
      if constexpr (!BWD)
        publish<2>(&bo[nt][hf], u[nt][0], u[nt][1], scale_of(column_max(abs_max2(u[nt]))), lane);
#pragma unroll
      for (int x = 0; x < 2; ++x) u[nt][x] *= gt.out[x];
      publish<2>(&bu[nt][hf], u[nt][0], u[nt][1], scale_of(column_max(abs_max2(u[nt]))), lane);
    }
    if constexpr (!BWD) {
      load_tri(xa, c.xa, next);
    } else {
      // what the gradient needs of this chunk
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (!in[nt]) continue;
#pragma unroll
        for (int i = 0; i < MW; ++i)
          store_tile(c.states + hid * DP * c.dvp + 16 * nt, 16 * (hf * MW + i), c.dvp, soff,
                     s[nt][i]);
#pragma unroll
        for (int x = 0; x < 2; ++x)
          store_tile(c.e + hid * kChunk * c.dvp + 16 * nt, 16 * (2 * hf + x), c.dvp, soff,
                     e[nt][x]);
      }
    }
    exchange();
    // S <- exp(G_64) S + K^T (exp(G_64 - G) o U)
    if constexpr (BWD) load_tri(xa, c.xa, next);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      half8 f[2][2];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int y = 0; y < 2; ++y) f[ks][y] = bu[nt][ks].f[y][lane];
      const float i0 = gt.kinv * bu[nt][0].inv[m], i1 = gt.kinv * bu[nt][1].inv[m];
#pragma unroll
      for (int i = 0; i < MW; ++i) {
        f32x4 acc[2] = {};
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) acc[ks] = mfma_pieces<NP, 2>(kt[i][ks], f[ks], acc[ks]);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          s[nt][i][r] = fmaf(gt.total, s[nt][i][r], fmaf(i0, acc[0][r], i1 * acc[1][r]));
      }
    }
    load_kt(next);
    if constexpr (!BWD) {
      // O = scale exp(G) o (Q S) + P U
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        f32x4 acc[2][2] = {};
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          if (ks > hf) break;
          const half8 f[2] = {bo[nt][ks].f[0][lane], bo[nt][ks].f[1][lane]};
#pragma unroll
          for (int x = 0; x < 2; ++x) acc[x][ks] = mfma_pieces<2, 2>(pa[x][ks], f, acc[x][ks]);
        }
        const float i0 = gt.pinv * bo[nt][0].inv[m], i1 = gt.pinv * bo[nt][1].inv[m];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int r = 0; r < 4; ++r) o[nt][x][r] += fmaf(i0, acc[x][0][r], i1 * acc[x][1][r]);
      }
      rows_o.store(o, chunk, len, a.l, whole, ok, hf, q);
      load_tri(pa, c.pa, next);
    }
    gt = gn;
  }
  if constexpr (!BWD) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (!ok[nt]) continue;
#pragma unroll
      for (int i = 0; i < MW; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * (hf * MW + i) + 4 * q + r;
          if (row < a.dk) a.s1[(p.head * a.dk + row) * a.dv + p.col0 + 16 * nt] = s[nt][i][r];
        }
      // outputs past the last live chunk
      for (int64_t t = (int64_t)chunks * kChunk + 4 * hf + q; t < a.l; t += 8)
        store1<T>(a.o, ((p.b * a.l + t) * a.hv + p.h) * a.dv + p.col0 + 16 * nt, 0.f);
    }
  }
}

// With W = dL/dU in full, dS the gradient of the state after the chunk:
//   dU = P^T dO + exp(G_64 - G) o (K dS),   W = dU - X^T (beta o dU),
//   dV = beta o W,
//   dS <- exp(G_64) dS + Q^T (scale exp(G) o dO) - K^T (exp(G) o dV).
template <int T, int DP, int NT, int NC>
__device__ __forceinline__ void scan_back(const ChunkArgs& c, int block, int blocks, char* lds) {
  constexpr int NP = T == T_F32 ? 2 : 1;
  constexpr int KS = DP / 32, MT = DP / 16, MW = MT / 2;
  typedef Raw<T> R;
  auto& [bs, by, bu, bo, bd] = ((BlocksBack<KS, NT>*)lds)[uniform((int)threadIdx.x >> 7)];
  const DeltaArgs& a = c.a;
  const Place p = place_of<NT, NC>(c, block, blocks);
  const int lane = threadIdx.x & 63, hf = uniform((int)threadIdx.x >> 6) & 1;
  const int m = lane & 15, q = lane >> 4;
  const int64_t len = live_tokens(a, p.b);
  const int chunks = (int)((len + kChunk - 1) / kChunk);
  const uint32_t loff = 16 * lane, soff = 4 * (4 * q * c.dvp + p.col0);
  const bool whole = p.block + 16 * NT <= a.dv;  // no column past the head size
  bool ok[NT], in[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    ok[nt] = p.col0 + 16 * nt < a.dv;
    in[nt] = p.block + 16 * nt < c.dvp;
  }
  f32x4 s[NT][MW];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < MW; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * (hf * MW + i) + 4 * q + r;
        s[nt][i][r] = a.ds1 && ok[nt] && row < a.dk
                          ? a.ds1[(p.head * a.dk + row) * a.dv + p.col0 + 16 * nt] : 0.f;
      }

  half8 ka[2][KS][NP], kt[MW][2][NP], qt[MW][2][NP], xt[2][2][2], pt[2][2][2];
  typename R::type dr[NT][2][4];
  Gates gt, gn;
  const auto kid_of = [&](int chunk) { return (p.b * c.nc + chunk) * a.hk + p.hk; };
  const auto hid_of = [&](int chunk) { return (p.b * c.nc + chunk) * a.hv + p.h; };
  const auto load_ka = [&](int chunk) {
    const Frag* src = c.ka + kid_of(chunk) * NP * 4 * KS * 64;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int y = 0; y < NP; ++y)
          ka[x][ks][y] = at_lane(src + ((y * 4 + 2 * hf + x) * KS + ks) * 64, loff);
  };
  const auto load_t = [&](half8(&f)[MW][2][NP], const Frag* base, int chunk) {
    const Frag* src = base + kid_of(chunk) * NP * MT * 2 * 64;
#pragma unroll
    for (int i = 0; i < MW; ++i)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int y = 0; y < NP; ++y)
          f[i][ks][y] = at_lane(src + ((y * MT + hf * MW + i) * 2 + ks) * 64, loff);
  };
  // rows 32..63 of an upper triangular operand have their second block only
  const auto load_tri = [&](half8(&f)[2][2][2], const Frag* base, int chunk) {
    const Frag* src = base + hid_of(chunk) * 2 * kTri * 64;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int y = 0; y < 2; ++y)
          if (ks == 1 || !hf)
            f[x][ks][y] = at_lane(src + (y * kTri + (hf ? 4 + x : 2 * x + ks)) * 64, loff);
  };
  const Rows<T, NT> rows_d(a.dout, a.do_stride, p, hf, q),
      rows_dv(a.dv_out, a.l, a.hv, a.dv, p, hf, q);
  const auto load_d = [&](int chunk) { rows_d.load(dr, chunk, len, whole, ok, hf, q); };
  if (chunks > 0) {
    const int last = chunks - 1;
    gt.load(c.gate + hid_of(last), hf, q);
    load_d(last);
    load_ka(last);
    load_tri(pt, c.pt, last);
    load_tri(xt, c.xt, last);
    load_t(kt, c.kt, last);
    load_t(qt, c.qt, last);
  }
  for (int chunk = chunks - 1; chunk >= 0; --chunk) {
    const int next = chunk > 0 ? chunk - 1 : 0;
    const int64_t hid = hid_of(chunk);
    gn.load(c.gate + hid_of(next), hf, q);
    f32x4 d[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const Scale ss = scale_of(column_max(abs_max(s[nt])));
#pragma unroll
      for (int i = 0; i < MW; i += 2)
        publish<2>(&bs[nt][(hf * MW + i) / 2], s[nt][i], s[nt][i + 1], ss, lane);
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int r = 0; r < 4; ++r) d[nt][x][r] = R::value(dr[nt][x][r]);
      publish<NP>(&bd[nt][hf], d[nt][0], d[nt][1], scale_of(column_max(abs_max2(d[nt]))), lane);
    }
    load_d(next);
    exchange();
    f32x4 w[NT][2], y[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      f32x4 acc[2][2] = {}, acp[2][2] = {};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const half8 f[2] = {bs[nt][ks].f[0][lane], bs[nt][ks].f[1][lane]};
#pragma unroll
        for (int x = 0; x < 2; ++x)
          acc[x][ks / (KS / 2)] = mfma_pieces<NP, 2>(ka[x][ks], f, acc[x][ks / (KS / 2)]);
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (ks < hf) continue;
        half8 f[NP];
#pragma unroll
        for (int z = 0; z < NP; ++z) f[z] = bd[nt][ks].f[z][lane];
#pragma unroll
        for (int x = 0; x < 2; ++x) acp[x][ks] = mfma_pieces<2, NP>(pt[x][ks], f, acp[x][ks]);
      }
      const float i0 = gt.kinv * bs[nt][0].inv[m], i1 = gt.kinv * bs[nt][KS - 1].inv[m];
      const float p0 = gt.pinv * bd[nt][0].inv[m], p1 = gt.pinv * bd[nt][1].inv[m];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          w[nt][x][r] = fmaf(gt.out[x][r], fmaf(i0, acc[x][0][r], i1 * acc[x][1][r]),
                             fmaf(p0, acp[x][0][r], p1 * acp[x][1][r]));
        y[nt][x] = gt.beta[x] * w[nt][x];
      }
      publish<2>(&by[nt][hf], y[nt][0], y[nt][1], scale_of(column_max(abs_max2(y[nt]))), lane);
    }
    // the state's gradient after this chunk, while the exchange is under way
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (!in[nt]) continue;
#pragma unroll
      for (int i = 0; i < MW; ++i)
        store_tile(c.dstates + hid * DP * c.dvp + 16 * nt, 16 * (hf * MW + i), c.dvp, soff,
                   s[nt][i]);
    }
    exchange();
    f32x4 g[NT][2];
    load_ka(next);
    load_tri(pt, c.pt, next);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      f32x4 acc[2][2] = {};
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (ks < hf) continue;
        const half8 f[2] = {by[nt][ks].f[0][lane], by[nt][ks].f[1][lane]};
#pragma unroll
        for (int x = 0; x < 2; ++x) acc[x][ks] = mfma_pieces<2, 2>(xt[x][ks], f, acc[x][ks]);
      }
      const float i0 = gt.xinv * by[nt][0].inv[m], i1 = gt.xinv * by[nt][1].inv[m];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int r = 0; r < 4; ++r) w[nt][x][r] -= fmaf(i0, acc[x][0][r], i1 * acc[x][1][r]);
        y[nt][x] = gt.beta[x] * w[nt][x];
        g[nt][x] = y[nt][x];
        y[nt][x] *= -gt.kpart * gt.into[x];
        d[nt][x] *= a.scale * gt.qpart * gt.into[x];
        if (in[nt])
          store_tile(c.dw + hid * kChunk * c.dvp + 16 * nt, 16 * (2 * hf + x), c.dvp, soff,
                     w[nt][x]);
      }
      // one scale for both operands, so that one sum takes both products; of
      // K's and Q's own scales they take what the two differ by
      const Scale ys = scale_of(column_max(fmaxf(abs_max2(y[nt]), abs_max2(d[nt]))));
      publish<2>(&bu[nt][hf], y[nt][0], y[nt][1], ys, lane);
      publish<2>(&bo[nt][hf], d[nt][0], d[nt][1], ys, lane);
    }
    rows_dv.store(g, chunk, len, a.l, whole, ok, hf, q);
    exchange();
    load_tri(xt, c.xt, next);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      half8 f[2][2], g[2][2];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          f[ks][z] = bu[nt][ks].f[z][lane];
          g[ks][z] = bo[nt][ks].f[z][lane];
        }
      const float i0 = gt.top * bu[nt][0].inv[m], i1 = gt.top * bu[nt][1].inv[m];
#pragma unroll
      for (int i = 0; i < MW; ++i) {
        f32x4 acc[2] = {};
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          acc[ks] = mfma_pieces<NP, 2>(kt[i][ks], f[ks], acc[ks]);
          acc[ks] = mfma_pieces<NP, 2>(qt[i][ks], g[ks], acc[ks]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
          s[nt][i][r] = fmaf(gt.total, s[nt][i][r], fmaf(i0, acc[0][r], i1 * acc[1][r]));
      }
    }
    load_t(kt, c.kt, next);
    load_t(qt, c.qt, next);
    gt = gn;
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    if (!ok[nt]) continue;
    if (a.ds0) {
#pragma unroll
      for (int i = 0; i < MW; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * (hf * MW + i) + 4 * q + r;
          if (row < a.dk) a.ds0[(p.head * a.dk + row) * a.dv + p.col0 + 16 * nt] = s[nt][i][r];
        }
    }
    for (int64_t t = (int64_t)chunks * kChunk + 4 * hf + q; t < a.l; t += 8)
      store1<T>(a.dv_out, ((p.b * a.l + t) * a.hv + p.h) * a.dv + p.col0 + 16 * nt, 0.f);
  }
}

template <int T, int DP, int NT, int NC>
__global__ void __launch_bounds__(128 * NC) delta_scan(ChunkArgs c) {
  extern __shared__ __align__(16) char lds[];
  scan<T, DP, NT, NC, false>(c, (int)blockIdx.x, (int)gridDim.x, lds);
}

// The states again and their gradients: neither needs the other, so half of
// the workgroups do the one and half the other, which few heads leave room
// for (2x700 tokens of 8 heads, 64x64, fp32: 36 us together, 26 + 36 one after
// the other; 8x2048 tokens of 16 heads, bf16, fill the device with either).
template <int T, int DP, int NT, int NC>
__global__ void __launch_bounds__(128 * NC) delta_scan_bwd(ChunkArgs c) {
  extern __shared__ __align__(16) char lds[];
  const int blocks = (int)(gridDim.x / 2), block = (int)blockIdx.x;
  if (block < blocks) scan_back<T, DP, NT, NC>(c, block, blocks, lds);
  else scan<T, DP, NT, NC, true>(c, block - blocks, blocks, lds);
}

template <int T, int DP, int NT, int NC>
hipError_t go_nt(const ChunkArgs& c, bool bwd, hipStream_t st) {
  constexpr int KS = DP / 32;
  const int groups = (c.dvp / 16 + NT * NC - 1) / (NT * NC);
  const dim3 grid((uint32_t)(c.a.b * c.a.hv * groups * (bwd ? 2 : 1))), block(128 * NC);
  auto* f = bwd ? &delta_scan_bwd<T, DP, NT, NC> : &delta_scan<T, DP, NT, NC>;
  // (what a backward scan keeps is more than what recomputed states need)
  const int bytes =
      NC * (int)(bwd ? sizeof(BlocksBack<KS, NT>) : sizeof(Blocks<KS, NT, false>));
  if (bytes > 64 * 1024) {  // more than a launch may ask for unasked
    const hipError_t err = hipFuncSetAttribute(reinterpret_cast<const void*>(f),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err != hipSuccess) return err;
  }
  hipLaunchKernelGGL(f, grid, block, bytes, st, c);
  return hipGetLastError();
}

template <int T, int DP>
hipError_t go(const ChunkArgs& c, bool bwd, hipStream_t st) {
  // 32 columns a wave and two pairs a workgroup read each fragment from L2 a
  // quarter as often (8x2048 tokens of 16 heads: states again in 215 us, 235
  // with one pair, 265 with 16 columns); one pair of 16 columns gives four
  // times the workgroups, which few heads need to reach the compute units
  // (and fp32 fragments of 128 dimensions leave no registers for 32)
  if constexpr (T != T_F32 || DP == 64) {
    if (c.a.b * c.a.hv * (c.dvp / 16) > 512) return go_nt<T, DP, 2, 2>(c, bwd, st);
  }
  return go_nt<T, DP, 1, 1>(c, bwd, st);
}

template <int T>
hipError_t go_dp(const ChunkArgs& c, bool bwd, hipStream_t st) {
  return c.a.dk <= 64 ? go<T, 64>(c, bwd, st) : go<T, 128>(c, bwd, st);
}

inline hipError_t go_type(const ChunkArgs& c, bool bwd, hipStream_t st) {
  if (c.a.type == T_F32) return go_dp<T_F32>(c, bwd, st);
  if (c.a.type == T_BF16) return go_dp<T_BF16>(c, bwd, st);
  return go_dp<T_F16>(c, bwd, st);
}

}  // namespace scans

hipError_t launch_delta_scan(const ChunkArgs& c, bool bwd, hipStream_t st) {
  return scans::go_type(c, bwd, st);
}

}  // namespace seq
}  // namespace dwc
