// Matrix products with the elementwise part of a layer in their epilogue
// (sm_100a, tcgen05): none of the products below leaves an intermediate in
// memory that the next kernel would read back, and none is rounded before the
// epilogue has used it.
//   linear      C  = R + drop(act(A W^T + bias)),  Z = A W^T + bias kept on request
//   linear_bwd  dZ = drop(dY W) act'(Z),  db_j = sum over rows of dZ_j
//   gated       h  = act(x Wg^T) (x Wu^T),  [gate | up] kept on request
//   gated_bwd   dh = dy Wd;  dgate = dh up act'(gate),  dup = dh act(gate),  h = act(gate) up
//
// Structure (persistent over output tiles):
//   warp 0      TMA producer: fills a ring of shared-memory stages
//   warp 1      MMA issuer: one lane issues tcgen05.mma on 128 x bn x 16
//               (256 x bn x 16 for a pair of CTAs)
//   warps 2..9  epilogue: tcgen05.ld from tensor memory, elementwise, store
//               (4..11 where sums are held in registers, see CHUNK_MOST)
// The accumulator is double-buffered in tensor memory (2 x 256 columns), so the
// epilogue of one tile runs under the main loop of the next.
//
// The gated product is one product whose B tile holds bn / 2 rows of Wg and
// the same bn / 2 rows of Wu: gate and up of an element land in the same lane
// of tensor memory, bn / 2 columns apart. In a pair of CTAs the first stages
// the rows of Wg and the second those of Wu.
//
// What bounds them: a pair's k-block of 256 x 256 x 64 takes 512 cycles on the
// tensor cores, in which each SM fetches 32 KB (the L2 gives an SM about 60
// bytes a cycle) and moves 64 KB through its shared memory, whose 128 bytes a
// cycle are so nearly used up that each byte the epilogue moves there costs
// time. Measured at 16384 x 5504 x 2048 on one B200, interleaved with a library's
// plain product at 248 us: 251 us with a bias alone, 273 us with GELU and the
// pre-activation kept, 310 us for the backward step with the bias gradient;
// 8192 x 13824 x 5120 gated, the halves kept, 1512 us (1534 TFLOP/s) beside 1638.
// Back to back for long, the card's power limit holds all of them to about 1390
// TFLOP/s.
#include <type_traits>

#include "act_dropout.cuh"

namespace mt {

namespace {

constexpr int BM = 128;
constexpr int BK = 64;       // 64 bf16 = 128 bytes: one swizzle row
constexpr int GROUP_M = 16;  // tile raster: 16 M-tiles share a band of N-tiles

// Each epilogue warp's staging buffer: a block of 32 rows x 32 columns of fp32.
constexpr int EPI_BYTES = 4096;

enum Epi : int { E_LINEAR_BF16, E_LINEAR_F32, E_BWD, E_GATED, E_GATED_BWD };

// Epilogue warps: two to a lane quarter, each taking one half of a tile's blocks
// of 32 columns.
constexpr int EPI_WARPS = 8;

// The tensor core adds a step of 16 products to its accumulator by truncation:
// a sum comes out low by about 9.5e-10 K of itself. Beside a bf16 output's
// rounding that is nothing, but fp32 outputs (a residual stream, the bias
// gradient) would show it: 2e-6 at K = 2048, 6e-6 at 5504, where one in fp32
// registers is off by under 1e-6. So from K = 897 on their kernels accumulate a
// chunk of the k-blocks at a time and add the chunks in the epilogue warps'
// registers (CHUNKED). Measured on one B200, interleaved, plain -> chunked: error
// 6.0e-6 -> 8.6e-7 and 265 -> 293 us for dropout and an fp32 residual at 16333 x
// 2048 x 5504; the bias gradient's 2.1e-6 -> 8.9e-7 and 286 -> 310 us at 16384 x
// 5504 x 2048.
constexpr int CHUNK_MOST = 14;  // k-blocks of a K that is accumulated at once
constexpr bool may_chunk(int epi) { return epi == E_LINEAR_F32 || epi == E_BWD; }

// Their 128 sums a thread do not fit the 168 registers of ten or twelve warps,
// so the copy and MMA warps fill a warpgroup of four (two of them idle) that
// gives registers to the eight epilogue warps: 56 x 128 + 224 x 256 = 168 x 384.
template <bool CHUNKED>
struct Warps {
  static constexpr int FIRST = CHUNKED ? 4 : 2;  // the first epilogue warp
  static constexpr int THREADS = 32 * (FIRST + EPI_WARPS);
  static constexpr int FEW = 56, MANY = 224;
};
constexpr int SMEM_MOST = 232448;  // 227 KB
constexpr int BAR_BYTES = 256;     // barriers of at most 12 stages
constexpr int MAX_STAGES = 12;
constexpr uint32_t TMEM_COLS = 512;  // two accumulators of up to 256 columns

// What the epilogue reads beside the accumulator (R, Z, gate and up) is
// fetched DEPTH blocks ahead: a block's share is 2 KB to a warp, or 4 KB.
template <int EPI>
struct Ahead {
  static constexpr int BLOCK = EPI == E_GATED ? 0 : EPI == E_LINEAR_BF16 || EPI == E_BWD ? 2048 : 4096;
  static constexpr int DEPTH = BLOCK == 0 ? 1 : 4096 / BLOCK;
};

// The tile and the pipeline of a launch, chosen by the host. A tile is 128
// rows (256 for a pair of CTAs) by bn columns. A stage holds `sub` k-blocks of
// a_rows rows of A and b_rows of B, 64 deep: several where they are small, so
// that a barrier is passed for 16 KB or more and rows are read 128 sub bytes at
// a time.
struct Tile {
  int bn, a_rows, b_rows, sub, stages;
  // The full-width pair kernel only: the first `whole` tiles fill whole waves;
  // each of the rest is cut into `split` narrower ones (1, 2 or 4), so that the
  // last wave is shared by more pairs.
  int whole, split;
  // k-blocks of an accumulation, multiples of sub: the first two chunks of a
  // tile, which run while the epilogue warps finish the tile before, and the
  // others.
  int chunk_first, chunk_rest;
};

struct Params {
  Tile t;
  int M, N, K;  // N: columns of the output (of each of gate and up)
  int act;
  DropDesc drop;
  const bf16* bias;
  const void* R;
  int64_t ldr;
  bf16* Z;  // linear: written; linear_bwd: read
  int64_t ldz;
  void* C;
  int64_t ldc;
  bf16* gu;  // gated: written (NULL: not kept); gated_bwd: read
  int64_t ldgu;
  bf16* dgu;  // gated_bwd
  int64_t lddgu;
  float* part;  // linear_bwd: sums over 32 rows, [ceil(M / 32), N rounded up to 4]; NULL: none
  int* err;
  uint64_t wait_ns;  // limit of the single-CTA form's main-loop waits; 0: give up at the first incomplete poll
};

__device__ __forceinline__ void tile_coords(int tile, int num_m, int num_n, int& mb, int& nb) {
  const int per_group = GROUP_M * num_n;
  const int g = tile / per_group;
  const int first_m = g * GROUP_M;
  const int gsize = min(num_m - first_m, GROUP_M);
  const int r = tile - g * per_group;
  mb = first_m + r % gsize;
  nb = r / gsize;
}

// ---------------------------------------------------------------------------
// Epilogues, one warp on 32 rows x 32 columns at a time. tcgen05.ld gives a
// lane a whole row; storing from there would touch 32 lines with each
// instruction. So the block goes through shared memory, and each lane handles
// 16 bytes of a row beside its neighbours: 8 columns of the rows lane / 4 + 8 i
// where the output is bf16, 4 columns of the rows lane / 8 + 4 i where it is
// fp32 (with 8 columns there, each access would take half of every sector).
// ---------------------------------------------------------------------------

// 16-byte unit u of row r of an fp32 block is kept at u ^ (r % 8), so that
// neither the row-wise writes nor the reads below meet in a bank.
__device__ __forceinline__ void stage_f32(float* st, int lane, const uint32_t (&a)[32]) {
#pragma unroll
  for (int u = 0; u < 8; ++u)
    reinterpret_cast<uint4*>(st)[lane * 8 + (u ^ (lane & 7))] =
        make_uint4(a[4 * u], a[4 * u + 1], a[4 * u + 2], a[4 * u + 3]);
}
// W columns of row r, the piece'th from the block's left.
template <int W>
__device__ __forceinline__ void staged_f32(const float* st, int r, int piece, float (&v)[W]) {
#pragma unroll
  for (int h = 0; h < W / 4; ++h) {
    const float4 a = reinterpret_cast<const float4*>(st)[r * 8 + ((W / 4 * piece + h) ^ (r & 7))];
    v[4 * h] = a.x, v[4 * h + 1] = a.y, v[4 * h + 2] = a.z, v[4 * h + 3] = a.w;
  }
}
// The same for a block of bf16, 64 bytes to a row: unit u at u ^ (r / 2 % 4).
__device__ __forceinline__ void stage_bf16(uint4* st, int lane, const float (&v)[32]) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float w[8] = {v[8 * u],     v[8 * u + 1], v[8 * u + 2], v[8 * u + 3],
                        v[8 * u + 4], v[8 * u + 5], v[8 * u + 6], v[8 * u + 7]};
    st[lane * 4 + (u ^ ((lane >> 1) & 3))] = pack8(w);
  }
}
__device__ __forceinline__ uint4 staged_bf16(const uint4* st, int r, int u) { return st[r * 4 + (u ^ ((r >> 1) & 3))]; }

// How a lane's 32 elements of a block lie: NC columns of NR rows, STEP apart.
template <int EPI>
struct Lay {
  static constexpr int NC = EPI == E_LINEAR_F32 ? 4 : 8, NR = 32 / NC, LANES = 32 / NC, STEP = 32 / LANES;
  static __device__ __forceinline__ int row(int lane) { return lane / LANES; }
  static __device__ __forceinline__ int col(int lane) { return lane % LANES * NC; }
};

// What a lane reads beside the accumulator: R, Z, or gate and up.
struct Aux {
  uint4 x[8];
};

// Eight bf16 of which n exist, as they are stored; zeros behind them.
__device__ __forceinline__ uint4 load8_raw(const bf16* p, int n) {
  if (n >= 8) return *reinterpret_cast<const uint4*>(p);
  float t[8];
  load_n<8>(p, n, t);
  return pack8(t);
}

template <int EPI>
__device__ __forceinline__ bool reads_aux(const Params& p) {
  return EPI == E_BWD ? p.act != MT_ACT_NONE : EPI == E_GATED_BWD ? true : EPI == E_GATED ? false : p.R != nullptr;
}
// Read where it is used, for a block that the matrix ends in.
template <int EPI>
__device__ __forceinline__ void load_aux(const Params& p, int row0, int col, int end, Aux& a) {
  using L = Lay<EPI>;
  const int n = end - col;
  if (!reads_aux<EPI>(p) || n <= 0) return;
#pragma unroll
  for (int i = 0; i < L::NR; ++i) {
    const int row = row0 + L::STEP * i;
    if (row >= p.M) break;
    if (EPI == E_LINEAR_BF16) {
      a.x[i] = load8_raw(reinterpret_cast<const bf16*>(p.R) + row * p.ldr + col, n);
    } else if (EPI == E_LINEAR_F32) {
      float t[4];
      load_n<4>(reinterpret_cast<const float*>(p.R) + row * p.ldr + col, n, t);
      a.x[i] = make_uint4(__float_as_uint(t[0]), __float_as_uint(t[1]), __float_as_uint(t[2]), __float_as_uint(t[3]));
    } else if (EPI == E_BWD) {
      a.x[i] = load8_raw(p.Z + row * p.ldz + col, n);
    } else {
      const bf16* g = p.gu + row * p.ldgu + col;  // N is a multiple of 8
      a.x[2 * i] = *reinterpret_cast<const uint4*>(g);
      a.x[2 * i + 1] = *reinterpret_cast<const uint4*>(g + p.N);
    }
  }
}

// The same for a block inside the matrix, ahead of time and into shared memory:
// a lane copies the very pieces that it reads back itself, so nothing but its
// own copies has to be waited for.
template <int EPI>
__device__ __forceinline__ void fetch_aux(const Params& p, uint32_t slot, int row0, int col) {
  using L = Lay<EPI>;
  if (!reads_aux<EPI>(p)) return;
#pragma unroll
  for (int i = 0; i < L::NR; ++i) {
    const int row = row0 + L::STEP * i;
    if (EPI == E_LINEAR_BF16) {
      copy16(slot + i * 512, reinterpret_cast<const bf16*>(p.R) + row * p.ldr + col);
    } else if (EPI == E_LINEAR_F32) {
      copy16(slot + i * 512, reinterpret_cast<const float*>(p.R) + row * p.ldr + col);
    } else if (EPI == E_BWD) {
      copy16(slot + i * 512, p.Z + row * p.ldz + col);
    } else {
      const bf16* g = p.gu + row * p.ldgu + col;
      copy16(slot + i * 1024, g);
      copy16(slot + i * 1024 + 512, g + p.N);
    }
  }
}
template <int EPI>
__device__ __forceinline__ void fetched_aux(const uint4* slot, Aux& a) {
#pragma unroll
  for (int i = 0; i < (EPI == E_LINEAR_BF16 || EPI == E_BWD ? 4 : 8); ++i) a.x[i] = slot[i * 32];
}

// The lane's part of the staged block; rows and columns outside the matrix
// hold what the product of zeros left there.
template <int EPI, int NR, int NC>
__device__ __forceinline__ void staged_rows(const float* st, int lane, float (&v)[NR][NC]) {
  using L = Lay<EPI>;
#pragma unroll
  for (int i = 0; i < NR; ++i) staged_f32<NC>(st, L::row(lane) + L::STEP * i, lane % L::LANES, v[i]);
}
template <int EPI, int NR, int NC>
__device__ __forceinline__ void drop_rows(const Params& p, const DropKey& key, int row0, int col, float (&v)[NR][NC]) {
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int h = 0; h < NC / 4; ++h)
      drop4(v[i] + 4 * h, (col >> 2) + h, p.drop.row0 + (uint32_t)(row0 + Lay<EPI>::STEP * i), p.drop, key);
}
template <int EPI, bool FULL, int NR, int NC, typename T>
__device__ __forceinline__ void store_rows(T* out, int64_t ld, int row0, int M, int n, const float (&v)[NR][NC]) {
  using L = Lay<EPI>;
#pragma unroll
  for (int i = 0; i < NR; ++i)
    if (FULL || row0 + L::STEP * i < M) store_n<NC>(out + i * L::STEP * ld, FULL ? NC : n, v[i]);
}

// FULL: the block lies inside the matrix, so that nothing is tested per element
// and the rows' instructions interleave.
template <int EPI, int ACT, bool FULL>
__device__ __forceinline__ void linear_block(const Params& p, const DropKey& key, int row0, int col, int end, int lane,
                                             const float* st, const Aux& a) {
  using L = Lay<EPI>;
  using T = std::conditional_t<EPI == E_LINEAR_F32, float, bf16>;
  constexpr int NR = L::NR, NC = L::NC;
  const int n = end - col;
  if (!FULL && n <= 0) return;
  float v[NR][NC];
  staged_rows<EPI>(st, lane, v);
  if (p.bias) {
    float bias[NC];
    load_n<NC>(p.bias + col, FULL ? NC : n, bias);
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int e = 0; e < NC; ++e) v[i][e] += bias[e];
  }
  if (p.Z) store_rows<EPI, FULL>(p.Z + row0 * p.ldz + col, p.ldz, row0, p.M, n, v);
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int e = 0; e < NC; e += 2) {
      const float2 a2 = act_value<ACT>(make_float2(v[i][e], v[i][e + 1]));
      v[i][e] = a2.x, v[i][e + 1] = a2.y;
    }
  if (p.drop.on) drop_rows<EPI>(p, key, row0, col, v);
  if (p.R) {
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      float t[NC];
      if constexpr (NC == 8) {
        unpack8(a.x[i], t);
      } else {
        t[0] = __uint_as_float(a.x[i].x), t[1] = __uint_as_float(a.x[i].y);
        t[2] = __uint_as_float(a.x[i].z), t[3] = __uint_as_float(a.x[i].w);
      }
#pragma unroll
      for (int e = 0; e < NC; ++e) v[i][e] += t[e];
    }
  }
  store_rows<EPI, FULL>(reinterpret_cast<T*>(p.C) + row0 * p.ldc + col, p.ldc, row0, p.M, n, v);
}

template <int ACT, bool FULL>
__device__ __forceinline__ void bwd_block(const Params& p, const DropKey& key, int row0, int col, int end, int lane,
                                          const float* st, const Aux& a) {
  const int n = end - col;
  float v[4][8];
  staged_rows<E_BWD>(st, lane, v);
  if (ACT != MT_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float t[8];
      unpack8(a.x[i], t);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 slope = act_slope<ACT>(make_float2(t[e], t[e + 1]));
        v[i][e] *= slope.x, v[i][e + 1] *= slope.y;
      }
    }
  }
  if (p.drop.on) drop_rows<E_BWD>(p, key, row0, col, v);  // last: a dropped element is 0 whatever Z holds there
  if (FULL || n > 0) store_rows<E_BWD, FULL>(reinterpret_cast<bf16*>(p.C) + row0 * p.ldc + col, p.ldc, row0, p.M, n, v);
  if (p.part) {
    float sum[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sum[e] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[e] += FULL || row0 + 8 * i < p.M ? v[i][e] : 0.f;
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], o);
    const int first = row0 - (lane >> 2);
    if (lane < 4 && (FULL || first < p.M)) {
      float* o = p.part + (int64_t)(first >> 5) * ((p.N + 3) & ~3) + col;  // rows of whole float4s
      if (FULL || n > 0) reinterpret_cast<float4*>(o)[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
      if (FULL || n > 4) reinterpret_cast<float4*>(o)[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
    }
  }
}

template <int ACT, bool FULL>
__device__ __forceinline__ void gated_bwd_block(const Params& p, int row0, int col, int end, int lane,
                                                const float* st, const Aux& a) {
  if (!FULL && col >= end) return;  // end is a multiple of 8
  float v[4][8];
  staged_rows<E_GATED_BWD>(st, lane, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = row0 + 8 * i;
    if (!FULL && row >= p.M) break;
    float g[8], u[8], h[8];
    unpack8(a.x[2 * i], g);
    unpack8(a.x[2 * i + 1], u);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      float2 value, slope;
      act_both<ACT>(make_float2(g[e], g[e + 1]), value, slope);
      h[e] = value.x * u[e], h[e + 1] = value.y * u[e + 1];
      g[e] = v[i][e] * u[e] * slope.x, g[e + 1] = v[i][e + 1] * u[e + 1] * slope.y;
      u[e] = v[i][e] * value.x, u[e + 1] = v[i][e + 1] * value.y;
    }
    bf16* o = p.dgu + row * p.lddgu + col;
    store8(o, g);
    store8(o + p.N, u);
    if (p.C) store8(reinterpret_cast<bf16*>(p.C) + row * p.ldc + col, h);
  }
}

// One block with its activation and fullness as constants.
template <int EPI, bool FULL>
__device__ __forceinline__ void block(const Params& p, const DropKey& key, int row0, int col, int end, int lane,
                                      const float* st, const Aux& a) {
  if constexpr (EPI == E_LINEAR_BF16 || EPI == E_LINEAR_F32)
    MT_WITH_ACT(p.act, (linear_block<EPI, ACT, FULL>(p, key, row0, col, end, lane, st, a)));
  if constexpr (EPI == E_BWD) MT_WITH_ACT(p.act, (bwd_block<ACT, FULL>(p, key, row0, col, end, lane, st, a)));
  if constexpr (EPI == E_GATED_BWD) MT_WITH_ACT(p.act, (gated_bwd_block<ACT, FULL>(p, row0, col, end, lane, st, a)));
}

// Gate and up meet in the registers of a row's lane; their bf16 blocks and h's
// go through shared memory to be stored.
template <int ACT>
__device__ __forceinline__ void gated_block(const Params& p, int row0, int col, int end, int lane, uint4* st,
                                            const uint32_t (&a)[32], const uint32_t (&b)[32]) {
  float v[32];
  const bool in = col < end;  // end is a multiple of 8
  uint4* st2 = st + 128;      // the second half of the warp's buffer
  if (p.gu) {
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(a[e]);
    stage_bf16(st, lane, v);
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(b[e]);
    stage_bf16(st2, lane, v);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = row0 + 8 * i, r = (lane >> 2) + 8 * i;
      if (!in || row >= p.M) break;
      bf16* o = p.gu + row * p.ldgu + col;
      *reinterpret_cast<uint4*>(o) = staged_bf16(st, r, lane & 3);
      *reinterpret_cast<uint4*>(o + p.N) = staged_bf16(st2, r, lane & 3);
    }
    __syncwarp();
  }
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const float2 h = act_value<ACT>(make_float2(__uint_as_float(a[e]), __uint_as_float(a[e + 1])));
    v[e] = h.x * __uint_as_float(b[e]), v[e + 1] = h.y * __uint_as_float(b[e + 1]);
  }
  stage_bf16(st, lane, v);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = row0 + 8 * i, r = (lane >> 2) + 8 * i;
    if (!in || row >= p.M) break;
    *reinterpret_cast<uint4*>(reinterpret_cast<bf16*>(p.C) + row * p.ldc + col) = staged_bf16(st, r, lane & 3);
  }
}

// A main-loop wait: with a limit of 0, one look at the barrier.
__device__ __forceinline__ bool wait_or_look(uint32_t bar, uint32_t parity, uint64_t limit) {
  return limit ? mbar_wait_u32(bar, parity, limit) : mbar_test(bar, parity);
}

// ---------------------------------------------------------------------------
// The kernel. PAIR: a cluster of two CTAs computes 256 rows with
// tcgen05.mma.cta_group::2; each stages its own 128 rows of A and half of B's
// rows, the leader (rank 0) issues the MMAs, both CTAs' copies complete on the
// leader's `full` barriers, the leader's commits release both CTAs' `empty`
// stages and both `tfull` accumulators, and both CTAs' epilogue warps release
// the leader's `tempty`. tmB2 is Wu's map for a gated product and unused
// otherwise.
// ---------------------------------------------------------------------------
template <bool PAIR, int EPI, bool WIDE, bool CHUNKED>
__global__ void __launch_bounds__(Warps<CHUNKED>::THREADS, 1)
    k_linear(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
             const __grid_constant__ CUtensorMap tmB2, const __grid_constant__ CUtensorMap tmS,
             const __grid_constant__ CUtensorMap tmS2, const __grid_constant__ Params p) {
  constexpr bool GATED = EPI == E_GATED;
  constexpr bool B_MN = EPI == E_BWD || EPI == E_GATED_BWD;  // B is stored [K, N]
  constexpr int TILE_M = PAIR ? 2 * BM : BM;
  using F = Ahead<EPI>;
  const int bn = WIDE ? 256 : p.t.bn, stages = p.t.stages;
  const int on = GATED ? bn / 2 : bn;  // output columns of a tile
  const int b_rows = WIDE ? (PAIR ? 128 : 256) : p.t.b_rows;
  const uint32_t a_bytes = (WIDE ? BM : p.t.a_rows) * (BK * 2), kb_bytes = a_bytes + b_rows * (BK * 2);
  const int sub = WIDE ? 1 : p.t.sub;
  const uint32_t stage_bytes = sub * kb_bytes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + stages * stage_bytes);
  uint64_t* empty = full + stages;
  uint64_t* tfull = empty + stages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  if (EPI == E_BWD) let_next_start();  // the column sums' kernel, which starts once all of these blocks have
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0;
  const uint64_t limit = PAIR ? kWaitLimitNs : p.wait_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], EPI_WARPS * (PAIR ? 2 : 1));
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    if (GATED) tma_prefetch_desc(&tmB2);
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(tmem_slot, TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, TMEM_COLS);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if (PAIR)
    cluster_sync();  // barrier initialisation and the allocation are visible to both CTAs
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int num_m = (p.M + TILE_M - 1) / TILE_M;
  const int num_n = (p.N + on - 1) / on;
  const int whole = WIDE ? p.t.whole : num_m * num_n, split = WIDE ? p.t.split : 1;
  const int num_tiles = whole + (num_m * num_n - whole) * split;
  // Tile index -> row block, first output column and output columns of the tile.
  auto tile_at = [&](int tile, int& mb, int& first, int& width) {
    const bool cut = WIDE && tile >= whole;
    const int u = tile - whole;
    int nb;
    tile_coords(cut ? whole + u / split : tile, num_m, num_n, mb, nb);
    width = cut ? on / split : on;
    first = nb * on + (cut ? u % split * width : 0);
  };
  const int num_kb = (p.K + BK - 1) / BK;
  constexpr int FIRST = Warps<CHUNKED>::FIRST;
  // The end of the chunk that begins at k-block kb0.
  auto chunk_end = [&](int kb0) {
    if (!CHUNKED) return num_kb;
    return min(num_kb, kb0 + (kb0 <= p.t.chunk_first ? p.t.chunk_first : p.t.chunk_rest));
  };
  const int first_tile = PAIR ? blockIdx.x >> 1 : blockIdx.x;
  const int tile_step = PAIR ? gridDim.x >> 1 : gridDim.x;

  if (warp < FIRST) {
    if (CHUNKED) lower_registers<Warps<CHUNKED>::FEW>();
    if (warp == 0) {
      // ---------------- TMA producer (the whole warp; one elected lane copies) ----------------
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;  // stages filled so far (for the teardown)
      const uint32_t fb0 = PAIR ? mapa_shared(smem_u32(&full[0]), 0) : 0;  // the leader's full barriers
      const uint32_t empty0 = smem_u32(&empty[0]);
      bool ok = true;
      for (int tile = first_tile; tile < num_tiles && ok; tile += tile_step) {
        int mb, first, width;
        tile_at(tile, mb, first, width);
        const int m0 = mb * TILE_M + (int)rank * BM;
        // A pair's B rows are split over its CTAs; a gated tile has one half from each weight.
        const int n0 = first + (PAIR && !GATED ? (int)rank * (width / 2) : 0);
        const bool cut = WIDE && width < on;  // tmS, tmS2: the same weights by fewer rows
        const CUtensorMap* mB = PAIR && GATED && rank ? (cut ? &tmS2 : &tmB2) : cut ? &tmS : &tmB;
        const int rows = cut ? b_rows / split : b_rows;
        const uint32_t bytes = a_bytes + rows * (BK * 2);
        for (int kb = 0; kb < num_kb; kb += sub) {
          const bool got = wait_or_look(empty0 + 8 * stage, phase ^ 1, limit);
          if (!__all_sync(0xffffffffu, got && !*abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + stage * stage_bytes;
          const int n = min(sub, num_kb - kb);  // k-blocks of this stage
          int k0 = kb * BK;
          if (elect_one()) {
            const uint32_t fb = fb0 + 8 * stage;
            if (!PAIR || rank == 0) mbar_arrive_expect_tx(&full[stage], (PAIR ? 2 : 1) * n * bytes);
            auto load = [&] {
              uint8_t* sb = sa + a_bytes;
              if (PAIR) {
                tma_load_2d_pair(sa, &tmA, fb, k0, m0);
                if (!B_MN) {
                  tma_load_2d_pair(sb, mB, fb, k0, n0);
                } else {
                  tma_load_2d_pair(sb, mB, fb, n0, k0);
                  if (rows > 64) tma_load_2d_pair(sb + 8192, mB, fb, n0 + 64, k0);
                }
              } else {
                tma_load_2d(sa, &tmA, &full[stage], k0, m0);
                if (GATED) {
                  tma_load_2d(sb, &tmB, &full[stage], k0, n0);
                  tma_load_2d(sb + (kb_bytes - a_bytes) / 2, &tmB2, &full[stage], k0, n0);
                } else if (!B_MN) {
                  tma_load_2d(sb, &tmB, &full[stage], k0, n0);
                } else {
#pragma unroll
                  for (int c = 0; c < 4; ++c)
                    if (c * 64 < b_rows) tma_load_2d(sb + c * 8192, &tmB, &full[stage], n0 + c * 64, k0);
                }
              }
            };
            load();
#pragma unroll 1
            for (int i = 1; i < n; ++i) {
              sa += kb_bytes, k0 += BK;
              load();
            }
          }
          ++issued;
          if (++stage == stages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok && lane == 0) {
        record_error(p.err, DEV_TIMEOUT_PRODUCER);
        *abort_flag = 1;
      }
      __syncwarp();
      if (lane == 0) {
        if (ok) {
          // Wait until the MMA has released every stage, so that no commit is on
          // its way to this CTA's barriers when it exits. If another role gives
          // up meanwhile, the MMA may never release them: drain the copies below.
          for (int i = 0; i < stages && ok; ++i) {
            const uint64_t t0 = globaltimer();
            while (!mbar_wait(&empty[stage], phase ^ 1, 0)) {
              if (!PAIR && *abort_flag) {
                ok = false;
                break;
              }
              if (globaltimer() - t0 > kWaitLimitNs) {
                record_error(p.err, DEV_TIMEOUT_TEARDOWN);
                *abort_flag = 1;
                ok = false;
                break;
              }
            }
            if (++stage == stages) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
        if (!ok && rank == 0) {
          // Every issued copy lands before the shared memory goes away: stage s
          // was last filled by fill s + STAGES q (the largest below `issued`), in
          // phase q mod 2. The leader's barriers count both CTAs' bytes.
          for (int s = 0; s < stages && s < issued; ++s) {
            const int q = (issued - 1 - s) / stages;
            if (!mbar_wait(&full[s], (uint32_t)(q & 1))) record_error(p.err, DEV_TIMEOUT_TEARDOWN);
          }
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      if (rank == 0) {
        // ---------------- MMA issuer ----------------
        // The whole warp walks the loop and one elected lane issues: with the
        // loop inside one lane's branch, every MMA and commit first moved its
        // operands to uniform registers, and a k-block took 560 cycles and more
        // to issue where the tensor core needs 512.
        const uint32_t idesc_whole = idesc_bf16_f32(TILE_M, bn, false, B_MN);
        const uint32_t idesc_cut = idesc_bf16_f32(TILE_M, bn / split, false, B_MN);
        // Descriptors of stage 0; stages and k-steps only move the start address.
        const uint32_t s0 = smem_u32(smem);
        const uint64_t a0 = sdesc_sw128(s0, 16, 1024);
        const uint64_t b0 = sdesc_sw128(s0 + a_bytes, B_MN ? 8192 : 16, 1024);
        const uint32_t kStage = stage_bytes >> 4, kBlock = kb_bytes >> 4;
        constexpr uint32_t kAStep = 32 >> 4, kBStep = (B_MN ? 2048 : 32) >> 4;
        const uint32_t full0 = smem_u32(&full[0]), empty0 = smem_u32(&empty[0]), tfull0 = smem_u32(&tfull[0]);
        int stage = 0;
        uint32_t phase = 0;
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        bool issued = false;
        for (int tile = first_tile, kb0 = 0; tile < num_tiles && ok;) {
          const bool free_acc = PAIR ? mbar_wait_cluster(&tempty[acc], acc_phase ^ 1)
                                     : wait_or_look(smem_u32(&tempty[acc]), acc_phase ^ 1, limit);
          if (!__all_sync(0xffffffffu, free_acc && !*abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + acc * 256;
          const uint32_t idesc = WIDE && tile >= whole ? idesc_cut : idesc_whole;
          const int kb1 = chunk_end(kb0);
          for (int kb = kb0; kb < kb1; kb += sub) {
            if (!__all_sync(0xffffffffu, wait_or_look(full0 + 8 * stage, phase, limit))) {
              ok = false;
              break;
            }
            // The stage's bytes were written by TMA and published through this
            // mbarrier, which orders them for the MMAs' reads: no tcgen05 fence.
            uint64_t ad = a0 + stage * kStage, bd = b0 + stage * kStage;
            const int n = min(sub, kb1 - kb);
            if (elect_one()) {
              auto multiply = [&](bool accumulate) {
#pragma unroll
                for (int kk = 0; kk < BK / 16; ++kk) {
                  if (PAIR)
                    umma_bf16_pair(d_tmem, ad + kk * kAStep, bd + kk * kBStep, idesc, accumulate || kk != 0);
                  else
                    umma_bf16(d_tmem, ad + kk * kAStep, bd + kk * kBStep, idesc, accumulate || kk != 0);
                }
              };
              multiply(kb != kb0);
#pragma unroll 1
              for (int i = 1; i < n; ++i) {
                ad += kBlock, bd += kBlock;
                multiply(true);
              }
              if (PAIR)
                umma_commit_both(empty0 + 8 * stage);
              else
                umma_commit_u32(empty0 + 8 * stage);
              if (kb + n == kb1) {
                if (PAIR)
                  umma_commit_both(tfull0 + 8 * acc);
                else
                  umma_commit_u32(tfull0 + 8 * acc);
              }
            }
            issued = true;
            if (++stage == stages) {
              stage = 0;
              phase ^= 1;
            }
          }
          if (!ok) break;
          if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1;
          }
          kb0 = kb1;
          if (kb1 == num_kb) kb0 = 0, tile += tile_step;
        }
        if (!ok && lane == 0) {
          record_error(p.err, DEV_TIMEOUT_MMA);
          *abort_flag = 1;
        }
        // Every MMA issued here completes before tensor memory is freed, also
        // when the epilogue gave up on an accumulator it will never read.
        if (issued) {
          if (elect_one()) {
            if (PAIR)
              umma_commit_pair(smem_u32(drain));
            else
              umma_commit(drain);
          }
          __syncwarp();
          if (!mbar_wait(drain, 0) && lane == 0) record_error(p.err, DEV_TIMEOUT_TEARDOWN);
        }
      }
    }
  } else {
    if (CHUNKED) raise_registers<Warps<CHUNKED>::MANY>();
    // ---------------- epilogue ----------------
    const int quarter = warp & 3;                // tensor-memory lanes this warp may read
    const int half = (warp - FIRST) >> 2;            // takes the first or the second half of the tile's blocks
    uint8_t* mine = smem + stages * stage_bytes + BAR_BYTES;
    float* st = reinterpret_cast<float*>(mine + (warp - FIRST) * EPI_BYTES);
    uint8_t* ahead = mine + EPI_WARPS * EPI_BYTES + (warp - FIRST) * F::DEPTH * F::BLOCK;
    const uint4* fetched = reinterpret_cast<uint4*>(ahead) + lane;
    const DropKey key = drop_key(p.drop);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int tile = first_tile; tile < num_tiles; tile += tile_step) {
      int mb, first, width;
      tile_at(tile, mb, first, width);
      const int row0 = mb * TILE_M + (int)rank * BM + quarter * 32 + Lay<EPI>::row(lane);  // this lane's first row
      // The warp's blocks; none (or less) in the second half of a tile of one
      // block and in a part of a tile that lies behind the last column.
      const int end = min(p.N, first + width), all = (end - first + 31) >> 5, first_half = (all + 1) >> 1;
      const int blocks = half ? all - first_half : first_half;
      const int share = half ? 32 * first_half : 0, col0 = first + share;
      const bool full_rows = mb * TILE_M + (int)rank * BM + quarter * 32 + 32 <= p.M;
      auto inside = [&](int k) { return full_rows && col0 + 32 * k + 32 <= end; };
      // One group of copies to a block, empty where there is nothing to copy.
      auto fetch = [&](int k) {
        if (F::BLOCK == 0) return;
        if (k < blocks && inside(k))
          fetch_aux<EPI>(p, smem_u32(fetched) + k % F::DEPTH * F::BLOCK, row0, col0 + 32 * k + Lay<EPI>::col(lane));
        copy_commit();
      };
#pragma unroll
      for (int k = 0; k < F::DEPTH; ++k) fetch(k);  // while the main loop runs
      // Waits for the next accumulator; warp-uniform outcome, for the tcgen05.ld
      // below is warp-collective.
      auto ready = [&] {
        if (__any_sync(0xffffffffu, *abort_flag) ||
            !__all_sync(0xffffffffu, wait_or_look(smem_u32(&tfull[acc]), acc_phase, limit))) {
          record_error(p.err, DEV_TIMEOUT_EPILOGUE);
          *abort_flag = 1;
          return false;
        }
        tc_fence_after();
        return true;
      };
      // Hands it back, once its last columns are in registers.
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR && rank)
            mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[acc]), 0));
          else
            mbar_arrive(&tempty[acc]);
        }
      };
      auto next = [&] {
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1;
        }
      };
      auto columns = [&](int k) {  // of block k in tensor memory
        return tmem_base + ((uint32_t)(quarter * 32) << 16) + acc * 256 + share + 32 * k;
      };
      // What becomes of block k once its sums are in registers.
      auto finish = [&](int k, const uint32_t(&a)[32]) {
        const int col = col0 + 32 * k + Lay<EPI>::col(lane);  // this lane's first column
        stage_f32(st, lane, a);
        __syncwarp();
        Aux aux;
        if (reads_aux<EPI>(p)) {  // its slots exist only then
          copy_wait<F::DEPTH - 1>();
          if (inside(k))
            fetched_aux<EPI>(fetched + k % F::DEPTH * (F::BLOCK / 16), aux);
          else
            load_aux<EPI>(p, row0, col, end, aux);
        }
        if (inside(k))
          block<EPI, true>(p, key, row0, col, end, lane, st, aux);
        else
          block<EPI, false>(p, key, row0, col, end, lane, st, aux);
        fetch(k + F::DEPTH);
        __syncwarp();  // the buffer is free for the next block
      };
      if constexpr (CHUNKED) {
        uint32_t sum[4][32];
        bool ok = true;
        for (int kb0 = 0; kb0 < num_kb; kb0 = chunk_end(kb0)) {
          if (!(ok = ready())) break;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k >= blocks) break;
            if (kb0 == 0) {
              tmem_ld_32x32b_x32(columns(k), sum[k]);
              tmem_ld_wait();
            } else {
              uint32_t a[32];
              tmem_ld_32x32b_x32(columns(k), a);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e)
                sum[k][e] = __float_as_uint(__uint_as_float(sum[k][e]) + __uint_as_float(a[e]));
            }
          }
          release();
          next();
        }
        if (!ok) break;
#pragma unroll 1
        for (int k = 0; k < blocks; ++k) {
          finish(k, sum[0]);
#pragma unroll
          for (int e = 0; e < 32; ++e) sum[0][e] = sum[1][e], sum[1][e] = sum[2][e], sum[2][e] = sum[3][e];
        }
      } else {
        if (!ready()) break;
        if (blocks <= 0) release();
#pragma unroll 1
        for (int k = 0; k < blocks; ++k) {
          uint32_t a[32];
          tmem_ld_32x32b_x32(columns(k), a);
          if constexpr (GATED) {
            uint32_t b[32];
            tmem_ld_32x32b_x32(columns(k) + width, b);
            tmem_ld_wait();
            if (k == blocks - 1) release();
            const int col = col0 + 32 * k + Lay<EPI>::col(lane);
            MT_WITH_ACT(p.act, (gated_block<ACT>(p, row0, col, end, lane, reinterpret_cast<uint4*>(st), a, b)));
            __syncwarp();  // the buffer is free for the next block
          } else {
            tmem_ld_wait();
            if (k == blocks - 1) release();
            finish(k, a);
          }
        }
        next();
      }
    }
    copy_wait<0>();  // also where the loop was left early
  }

  tc_fence_before();
  __syncwarp();
  if (PAIR)
    cluster_sync();  // no MMA of the pair and no tensor-memory read is outstanding
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem_base, TMEM_COLS);
    else
      tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
// What a launch needs: operands and the tile-independent parameters.
struct Op {
  const void* A;
  int64_t lda;
  const void* B;
  const void* B2;  // Wu of a gated product
  int64_t ldb;
  Params p;
};

// A k-block's cost to an SM: the larger of its MMAs (2 bn cycles for 128 rows, or
// for each half of a pair's 256) and of fetching its operands from L2 at about 60
// bytes a cycle, which is what bounds narrow tiles: 128 x 128 takes 546 cycles for
// 256 of MMA. In 60ths of a cycle.
int block_cost(int a_rows, int b_rows, int bn) {
  const int bytes = (a_rows + b_rows) * 128;
  return 2 * bn * 60 > bytes ? 2 * bn * 60 : bytes;
}

// The last wave of full-width pair tiles, `rest` of them for n pairs: cut in 1, 2
// or 4 (an MN-major operand comes in pieces of 64 columns: at most 2), whichever
// costs least. Measured on one B200, interleaved: the gated backward of 4099 x
// 1408 x 2048 (102 tiles: 74 whole, 28 cut in two) 38.1 us instead of 41.6, of
// 2048 x 5504 x 2048 61.9 instead of 71.5.
struct LastWave {
  int split;
  int64_t cost;
};
LastWave last_wave(int rest, int n, bool mn_major) {
  LastWave best{1, INT64_MAX};
  for (int s = 1; s <= (mn_major ? 2 : 4); s *= 2) {
    const int64_t c = (int64_t)((rest * s + n - 1) / n) * block_cost(BM, 128 / s, 256 / s);
    if (c < best.cost) best = LastWave{s, c};
  }
  return best;
}

// Chunks of the n k-blocks of a depth K, in stages of sub. One of c blocks loses up
// to 7e-8 c of itself (measured), so chunks c_i lose 7e-8 sum c_i^2 / (K / 64): a
// sum of 14.2 K / 64 at most keeps that below 1e-6. Up to 27 blocks that allows two
// halves, of which none is a stub. Beyond, the first two are as long as it allows
// (up to 20), for the tensor cores have nothing but those two to do while the
// epilogue warps finish the tile before; the rest have 12 at most.
struct Chunks {
  int first, rest;
};
Chunks chunks_of(int K, int sub) {
  const int n = (K + BK - 1) / BK;
  if (n <= 27) {
    const int half = ((n + 1) / 2 + sub - 1) / sub * sub;
    return Chunks{half, half};
  }
  auto whole = [&](int c) { return c > sub ? c / sub * sub : sub; };
  for (int first = 20; first > 12; --first) {
    const int left = n - 2 * first > 0 ? n - 2 * first : 0, second = n - first < first ? n - first : first;
    const int rest = left ? (left + (left + 11) / 12 - 1) / ((left + 11) / 12) : first;
    // left k-blocks in chunks of rest, the last one shorter
    const int full = left / rest, last = left - full * rest;
    const int lost = first * first + second * second + full * rest * rest + last * last;
    if (640 * (int64_t)lost <= 142 * (int64_t)K) return Chunks{whole(first), whole(rest)};
  }
  return Chunks{12, 12};
}

template <bool PAIR, int EPI, bool WIDE, bool CHUNKED>
int launch(Op o, int bn, int device, int num_sms, cudaStream_t st) {
  constexpr bool GATED = EPI == E_GATED, B_MN = EPI == E_BWD || EPI == E_GATED_BWD;
  constexpr int TILE_M = PAIR ? 2 * BM : BM;
  auto kernel = k_linear<PAIR, EPI, WIDE, CHUNKED>;
  Params& p = o.p;
  // Rows of A behind the last are not staged: an MMA then reads what lies
  // behind them in shared memory, and only its rows that are not stored see it.
  const int on = GATED ? bn / 2 : bn;
  p.t.bn = bn;
  p.t.a_rows = PAIR || p.M >= BM ? BM : (p.M + 7) / 8 * 8;
  p.t.b_rows = PAIR ? bn / 2 : bn;
  const bool aux = EPI == E_BWD ? p.act != MT_ACT_NONE : EPI == E_GATED_BWD ? true : EPI != E_GATED && p.R;
  const int epi = EPI_WARPS * (EPI_BYTES + (aux ? Ahead<EPI>::DEPTH * Ahead<EPI>::BLOCK : 0));
  const int kb_bytes = (p.t.a_rows + p.t.b_rows) * BK * 2;
  const int num_kb = (p.K + BK - 1) / BK;
  p.t.sub = kb_bytes > 16384 ? 1 : kb_bytes > 8192 ? 2 : 4;
  if (p.t.sub > num_kb) p.t.sub = num_kb;
  const int stage = p.t.sub * kb_bytes;
  // Without a bias gradient the backward's outputs are bf16 and need no chunks.
  if (CHUNKED) {  // multiples of sub, and num_kb > CHUNK_MOST
    const Chunks c = chunks_of(p.K, p.t.sub);
    p.t.chunk_first = c.first;
    p.t.chunk_rest = c.rest;
  }
  const int fit = (SMEM_MOST - 1024 - BAR_BYTES - epi) / stage;
  p.t.stages = fit < MAX_STAGES ? fit : MAX_STAGES;
  // An MMA on fewer staged rows of A still reads 16 KB from the stage's start.
  const int used = p.t.stages * stage + BAR_BYTES + epi, read = p.t.stages * stage - kb_bytes + BM * BK * 2;
  const int smem = 1024 + (used > read ? used : read);

  CUtensorMap ta, tb, tb2;
  bool ok = make_tensor_map_2d_bf16(&ta, o.A, p.K, p.M, o.lda, p.t.a_rows);
  const int b_box = GATED && !PAIR ? bn / 2 : p.t.b_rows;
  ok = ok && (B_MN ? make_tensor_map_2d_bf16(&tb, o.B, p.N, p.K, o.ldb, 64)
                   : make_tensor_map_2d_bf16(&tb, o.B, p.K, p.N, o.ldb, b_box));
  tb2 = tb;
  if (GATED) ok = ok && make_tensor_map_2d_bf16(&tb2, o.B2, p.K, p.N, o.ldb, b_box);
  if (!ok) return MT_ERR_ARG;

  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(Warps<CHUNKED>::THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  if (PAIR) {
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  // Per device, once: the shared-memory limit and the CTAs (pairs) that can be
  // resident together. Threads that race here write the same value.
  static int resident[kMaxDevices] = {};
  if (resident[device] == 0) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MOST) != cudaSuccess)
      return MT_ERR_CUDA;
    // The epilogue warps would wait for ever for registers that the block was not launched with.
    using W = Warps<CHUNKED>;
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess) return MT_ERR_CUDA;
    if (CHUNKED && fa.numRegs * W::THREADS < W::FEW * 32 * W::FIRST + W::MANY * 32 * EPI_WARPS) return MT_ERR_CONFIG;
    int r = PAIR ? num_sms / 2 : num_sms;
    if (PAIR) {
      int n = 0;
      cfg.gridDim = dim3(2 * r, 1, 1);
      if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0)
        r = n < r ? n : r;
      else
        cudaGetLastError();
    }
    resident[device] = r;
  }
  int64_t tiles = (int64_t)((p.M + TILE_M - 1) / TILE_M) * ((p.N + on - 1) / on);
  if (tiles > INT32_MAX / 8) return MT_ERR_ARG;
  p.t.whole = (int)tiles, p.t.split = 1;
  CUtensorMap ts = tb, ts2 = tb2;
  if (WIDE) {
    const int rest = (int)(tiles % resident[device]);
    p.t.split = tiles > rest ? last_wave(rest, resident[device], B_MN).split : 1;
    if (p.t.split > 1) {
      p.t.whole = (int)tiles - rest;
      tiles = p.t.whole + (int64_t)rest * p.t.split;
      if (!B_MN) ok = make_tensor_map_2d_bf16(&ts, o.B, p.K, p.N, o.ldb, p.t.b_rows / p.t.split);
      if (GATED) ok = ok && make_tensor_map_2d_bf16(&ts2, o.B2, p.K, p.N, o.ldb, p.t.b_rows / p.t.split);
      if (!ok) return MT_ERR_ARG;
    }
  }
  const int n = tiles < resident[device] ? (int)tiles : resident[device];
  cfg.gridDim = dim3(PAIR ? 2 * n : n, 1, 1);
  cudaLaunchKernelEx(&cfg, kernel, ta, tb, tb2, ts, ts2, p);
  return launch_status();
}

// The tile is the one whose waves cost least by block_cost().
template <int EPI>
int dispatch(const Op& o, cudaStream_t st) {
  int device = 0, sms = 0;
  if (cudaGetDevice(&device) != cudaSuccess || device >= kMaxDevices) return MT_ERR_CUDA;
  static int num_sms[kMaxDevices] = {};
  if (num_sms[device] == 0) {
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || sms <= 0)
      return MT_ERR_CUDA;
    num_sms[device] = sms;
  }
  sms = num_sms[device];
  constexpr bool B_MN = EPI == E_BWD || EPI == E_GATED_BWD;
  constexpr int G = EPI == E_GATED ? 2 : 1;  // a gated tile spends half of its columns on each of gate and up
  const int family = gemm_variant_now();
  int best = 0;
  bool best_pair = false;
  int64_t least = INT64_MAX;
  auto consider = [&](int bn, bool pair) {
    const int tm = pair ? 2 * BM : BM, tn = bn / G, n = pair ? sms / 2 : sms;
    const int64_t tiles = ((int64_t)o.p.M + tm - 1) / tm * ((o.p.N + tn - 1) / tn);
    const int each = block_cost(o.p.M < BM ? o.p.M : BM, pair ? bn / 2 : bn, bn);
    const int64_t cost = pair && bn == 256 && tiles > n ? tiles / n * each + last_wave((int)(tiles % n), n, B_MN).cost
                                                        : (tiles + n - 1) / n * each;
    // On a tie the wider tile, but single CTAs before pairs.
    if (cost < least || (cost == least && best_pair && !pair)) least = cost, best = bn, best_pair = pair;
  };
  // MN-major operands are staged 64 columns at a time; MMAs take widths of
  // multiples of 16 (a pair's of 32).
  if (family != 1)
    for (int bn = 256; bn >= (B_MN ? 128 : 64); bn -= B_MN ? 128 : 32) consider(bn, true);
  if (family != 2)
    for (int bn = 256; bn >= (B_MN ? 64 : 32); bn -= B_MN ? 64 : 16) consider(bn, false);
  if constexpr (may_chunk(EPI)) {
    // Without a bias gradient the backward's outputs are bf16 and need no chunks.
    if ((o.p.K + BK - 1) / BK > CHUNK_MOST && (EPI != E_BWD || o.p.part)) {
      if (best_pair && best == 256) return launch<true, EPI, true, true>(o, best, device, sms, st);
      return best_pair ? launch<true, EPI, false, true>(o, best, device, sms, st)
                       : launch<false, EPI, false, true>(o, best, device, sms, st);
    }
  }
  if (best_pair && best == 256) return launch<true, EPI, true, false>(o, best, device, sms, st);
  return best_pair ? launch<true, EPI, false, false>(o, best, device, sms, st)
                   : launch<false, EPI, false, false>(o, best, device, sms, st);
}

}  // namespace

int launch_linear_fwd(const LinearFwd& a, const DropDesc& drop, cudaStream_t st, int* dev_err) {
  Op o{};
  o.A = a.A, o.lda = a.lda, o.B = a.W, o.ldb = a.ldw;
  Params& p = o.p;
  p.M = a.M, p.N = a.N, p.K = a.K, p.act = a.act, p.drop = drop;
  p.bias = (const bf16*)a.bias, p.R = a.R, p.ldr = a.ldr, p.Z = (bf16*)a.Z, p.ldz = a.ldz, p.C = a.C, p.ldc = a.ldc;
  p.err = dev_err, p.wait_ns = gemm_wait_limit_now();
  return a.out_type == MT_F32 ? dispatch<E_LINEAR_F32>(o, st) : dispatch<E_LINEAR_BF16>(o, st);
}

size_t linear_bwd_partial_floats(int M, int N) { return (size_t)((M + 31) / 32) * ((N + 3) & ~3); }

int launch_linear_bwd_act(const LinearBwd& a, const DropDesc& drop, cudaStream_t st, int* dev_err) {
  Op o{};
  o.A = a.dY, o.lda = a.lddy, o.B = a.W, o.ldb = a.ldw;
  Params& p = o.p;
  p.M = a.M, p.N = a.N, p.K = a.K, p.act = a.act, p.drop = drop;
  p.Z = (bf16*)a.Z, p.ldz = a.ldz, p.C = a.dZ, p.ldc = a.lddz, p.part = a.db ? a.part : nullptr;
  p.err = dev_err, p.wait_ns = gemm_wait_limit_now();
  if (const int rc = dispatch<E_BWD>(o, st)) return rc;
  return a.db ? launch_column_sums(a.part, (a.M + 31) / 32, (a.N + 3) & ~3, a.N, a.db, a.N, nullptr, st) : MT_OK;
}

int launch_gated_ffn_fwd(const void* x, int64_t ldx, const void* Wgu, int64_t ldw, int act, void* gu, int64_t ldgu,
                         void* h, int64_t ldh, int M, int F, int K, cudaStream_t st, int* dev_err) {
  Op o{};
  o.A = x, o.lda = ldx, o.B = Wgu, o.B2 = (const bf16*)Wgu + (int64_t)F * ldw, o.ldb = ldw;
  Params& p = o.p;
  p.M = M, p.N = F, p.K = K, p.act = act, p.gu = (bf16*)gu, p.ldgu = ldgu, p.C = h, p.ldc = ldh;
  p.err = dev_err, p.wait_ns = gemm_wait_limit_now();
  return dispatch<E_GATED>(o, st);
}

int launch_gated_ffn_bwd(const void* dy, int64_t lddy, const void* Wd, int64_t ldw, const void* gu, int64_t ldgu,
                         int act, void* dgu, int64_t lddgu, void* h, int64_t ldh, int M, int F, int K, cudaStream_t st,
                         int* dev_err) {
  Op o{};
  o.A = dy, o.lda = lddy, o.B = Wd, o.ldb = ldw;
  Params& p = o.p;
  p.M = M, p.N = F, p.K = K, p.act = act, p.gu = (bf16*)gu, p.ldgu = ldgu, p.dgu = (bf16*)dgu, p.lddgu = lddgu;
  p.C = h, p.ldc = ldh, p.err = dev_err, p.wait_ns = gemm_wait_limit_now();
  return dispatch<E_GATED_BWD>(o, st);
}

}  // namespace mt
