// Attention of a few query tokens a sequence over the paged latent cache.
//
// All heads of a sequence attend to the same cached rows [c | k_r], and c is key and value
// at once, so the Sq * n_heads query rows of a sequence form the columns of one product
// per tile of 32 cached rows: S^T = [c | k_r] Q^T, then O^T += c^T P^T with c read
// transposed from the same LDS tile. A row is read from memory once for all heads.
//
// A wave owns 16 query rows: their operands (72 registers at latent 512) and their part of
// O (128) are what two waves a SIMD can hold. The eight waves of a workgroup are WQ groups
// of query rows x WT tiles worked on side by side x WD parts of the value width (the
// scores are then formed by each part), by the number of query rows.
//
// The work is the sequences' steps of 32 WT rows laid end to end, (sequence, block of query
// rows, step), cut into equal ranges for a fixed number of workgroups: ragged lengths
// balance without the host knowing them. A block of query rows whose steps fall into
// several ranges leaves its partial sums (O unnormalised, maximum, sum, all FP32) in the
// workspace, and a second kernel joins them in range order.
#include "latent.h"

namespace moe {
namespace {

constexpr int kTok = 32;        // cached rows a tile
constexpr int kAWaves = 8;
constexpr int kAThreads = kAWaves * kWave;
constexpr int kGroups = 256;    // workgroups: one a CU
constexpr int kMinSteps = 2;    // steps a range holds at least
constexpr int kAhead = 3;         // depth steps whose rows are read ahead
constexpr float kSlack = 8.0f;  // how far (log2) a score may pass the reference of its row

struct AbsorbedArgs {
  const uint16_t* q;
  const uint8_t* cache;
  const int32_t *table, *lengths;
  void* out;
  float* lse;
  int64_t* first;      // [B + 1]: steps before each sequence (one block of query rows)
  float* part;         // [kGroups][2] partial results
  int64_t n_pages, max_pages;
  int B, Sq, H, page, blocks;   // blocks of query rows a sequence
  float scale2;
  int out_bf16;
};

__device__ __forceinline__ f4 mfma16(bf8 a, bf8 b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ int length_of(const AbsorbedArgs& a, int b) {
  return (int)min((int64_t)max(a.lengths[b], 0), a.max_pages * a.page);
}
__device__ __forceinline__ int64_t range_steps(int64_t total) {
  return max((int64_t)kMinSteps, (total + kGroups - 1) / kGroups);
}
// floats of a partial result of n query rows: O, then the maxima and the sums
__host__ __device__ constexpr int64_t part_floats(int latent, int n) { return (int64_t)n * (latent + 2); }

// LDS tile of cached rows. Latent rows: 16-byte chunk c of row r at chunk c ^ latent_key(r)
// of its 256 bytes. A read of 16 rows at 4 chunks (ds_read_b128) is served in quarters of
// lanes 0-3, 12-15, 20-27 and the like: rows 0-3 and 12-15 of one chunk with rows 4-11 of
// the next; transposed reads take 8 rows at 2 adjacent chunks. With this key both touch
// each of the 64 banks once (with (r & 7) << 1 | r >> 3, quarters collided: a third of the
// LDS cycles).
__device__ __forceinline__ constexpr int latent_key(int r) {
  return (((r & 7) ^ ((r & 8) >> 1)) << 1) | ((r >> 3) & 1);
}
template <int R>
__device__ __forceinline__ int latent_off(int r, int c) { return r * 2 * R + ((c ^ latent_key(r)) << 4); }

template <int R>
struct __attribute__((aligned(256))) LatentTile {
  uint8_t c[kTok * 2 * R], r[kTok * 2 * kRope];
};

// Cache rows of a step staged by a wave, one row an instruction. A row that is not there
// (past the length, page out of range) is zero.
template <int R, int WT, bool FP8>
struct Stage {
  static constexpr int kRows = kTok * WT / kAWaves;
  u4 v[FP8 ? kRows : 1];
  float s[FP8 ? kRows : 1];
};

// The page of position pos of sequence b as the table has it (the table's last column for a
// position past it); a row number is formed from it a step later, when it has arrived.
__device__ __forceinline__ int page_of(const AbsorbedArgs& a, int b, int pos) {
  const int64_t p = min((int64_t)((uint32_t)pos / (uint32_t)a.page), a.max_pages - 1);
  return a.table[(int64_t)b * a.max_pages + p];
}
// The cache row of position pos, -1 if there is none.
__device__ __forceinline__ int row_slot(const AbsorbedArgs& a, int pg, int pos, int len) {
  const bool there = pos < len && pg >= 0 && pg < a.n_pages;
  return there ? pg * a.page + (int)((uint32_t)pos % (uint32_t)a.page) : -1;
}

// slots: lane j < kRows holds the cache row of the wave's j-th row.
template <int R, int WT, bool FP8>
__device__ __forceinline__ void load_rows(const AbsorbedArgs& a, Stage<R, WT, FP8>& g, LatentTile<R>* tiles, int slots,
                                          int wave, int lane) {
  constexpr int kRows = Stage<R, WT, FP8>::kRows, kBytes = cache_row_bytes(R, FP8);
  LatentTile<R>* t = tiles + wave * kRows / kTok;
  const int row0 = wave * kRows % kTok;
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int slot = __builtin_amdgcn_readlane(slots, j);
    const auto row = buffer_of(a.cache + (int64_t)max(slot, 0) * kBytes, slot >= 0 ? kBytes : 0);
    if constexpr (FP8) {
      // lanes of 16 codes, then 8 lanes of the rotary key; the lane's scale beside them
      g.v[j] = __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(row, lane * 16, 0, 0));
      g.s[j] = __builtin_bit_cast(
          float, __builtin_amdgcn_raw_buffer_load_b32(row, R + 2 * kRope + 4 * min(lane / 8, R / kTile - 1), 0, 0));
    } else {
      const int r = row0 + j;
      if (lane < R / 8) {
        const int c = (lane & ~15) | ((lane ^ latent_key(r)) & 15);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(row, (lds_byte*)(t->c + r * 2 * R), 16, c * 16, 0, 0, 0);
      }
    }
  }
  if constexpr (!FP8) {
    // rotary keys: lane l stages the 16 bytes at l * 16 of the wave's 128-byte rows
    if (lane < kRows * 8) {
      const int line = row0 / 2 + (lane >> 4);
      const int x = (lane & 15) ^ line_key(line);
      const int slot = __shfl(slots, 2 * line + (x >> 3) - row0);
      uint8_t* to = t->r + row0 * 128;
      if (slot >= 0)
        __builtin_amdgcn_global_load_lds(a.cache + (int64_t)slot * kBytes + 2 * R + (x & 7) * 16, (lds_byte*)to, 16, 0, 0);
      else
        *reinterpret_cast<u4*>(to + lane * 16) = u4{0, 0, 0, 0};
    }
  }
}

template <int R, int WT>
__device__ __forceinline__ void store_rows(const Stage<R, WT, true>& g, LatentTile<R>* tiles, int wave, int lane) {
  constexpr int kRows = Stage<R, WT, true>::kRows;
  LatentTile<R>* t = tiles + wave * kRows / kTok;
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int r = wave * kRows % kTok + j;
    if (lane < R / 16) {
      *reinterpret_cast<u4*>(t->c + latent_off<R>(r, 2 * lane)) = unpack_fp8(make_uint2(g.v[j][0], g.v[j][1]), g.s[j]);
      *reinterpret_cast<u4*>(t->c + latent_off<R>(r, 2 * lane + 1)) = unpack_fp8(make_uint2(g.v[j][2], g.v[j][3]), g.s[j]);
    } else if (lane < R / 16 + 8) {
      *reinterpret_cast<u4*>(t->r + tile_off<2 * kRope>(r, lane - R / 16)) = g.v[j];
    }
  }
}

// E4M3 rows by way of LDS (one tile a step): a wave copies its rows' codes there one step
// ahead of the conversion, so no register waits on memory across the products.
template <int R>
struct __attribute__((aligned(16))) CodeTile {
  uint8_t row[kTok][fp8_row_bytes(R)];
};

template <int R>
__device__ __forceinline__ void copy_codes(const AbsorbedArgs& a, CodeTile<R>* t, int slots, int wave, int lane) {
  constexpr int kRows = kTok / kAWaves, kBytes = fp8_row_bytes(R);
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int slot = __builtin_amdgcn_readlane(slots, j);
    const auto row = buffer_of(a.cache + (int64_t)max(slot, 0) * kBytes, slot >= 0 ? kBytes : 0);
    if (lane < kBytes / 16)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(row, (lds_byte*)t->row[wave * kRows + j], 16, lane * 16, 0, 0, 0);
  }
}

template <int R>
__device__ __forceinline__ void convert_codes(const CodeTile<R>& g, LatentTile<R>* t, int wave, int lane) {
  constexpr int kRows = kTok / kAWaves, kChunks = R / 16, kSide = kWave / kChunks;   // rows side by side
#pragma unroll
  for (int j = 0; j < kRows; j += kSide) {
    const int r = wave * kRows + j + lane / kChunks, c = lane % kChunks;
    const u4 v = *reinterpret_cast<const u4*>(g.row[r] + c * 16);
    const float s = *reinterpret_cast<const float*>(g.row[r] + R + 2 * kRope + 4 * (c / 8));
    *reinterpret_cast<u4*>(t->c + latent_off<R>(r, 2 * c)) = unpack_fp8(make_uint2(v[0], v[1]), s);
    *reinterpret_cast<u4*>(t->c + latent_off<R>(r, 2 * c + 1)) = unpack_fp8(make_uint2(v[2], v[3]), s);
  }
  if (lane < kRows * 8) {
    const int r = wave * kRows + lane / 8;
    *reinterpret_cast<u4*>(t->r + tile_off<2 * kRope>(r, lane % 8)) =
        *reinterpret_cast<const u4*>(g.row[r] + R + (lane % 8) * 16);
  }
}

template <int R, int WQ, int WT, int WD, bool FP8>
__global__ __launch_bounds__(kAThreads, 2) void absorbed_kernel(const AbsorbedArgs a) {
  static_assert(WQ * WT * WD == kAWaves, "waves");
  constexpr int kSteps = (R + kRope) / 32, kRows = kTok * WT / kAWaves, kStep = kTok * WT;
  constexpr int kCols = R / WD, kFrags = kCols / 16;   // kFrags is 4 or a multiple of 8
  constexpr int kQRows = 16 * WQ;
  // Query operands of the last kQLds steps wait in LDS where the registers do not hold all.
  constexpr int kQLds = kFrags == 32 ? 8 : 0;
  __shared__ LatentTile<R> tiles[2][WT];
  constexpr bool kCodes = FP8 && WT == 1;
  __shared__ CodeTile<kCodes ? R : 16> codes;
  __shared__ bf8 qlds[kAWaves][kQLds > 0 ? kQLds : 1][kWave];
  __shared__ int64_t wsum[kAWaves];
  __shared__ int64_t found[2];   // the sequence that holds the range's first step, its first step
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, grp = lane >> 4;
  const int wd = wave % WD, wt = wave / WD % WT, wq = wave / (WD * WT);

  // Steps before each sequence, twice: the total fixes the ranges, then the range's first
  // sequence is looked up.
  int64_t total = 0;
  for (int b = tid; b < a.B; b += kAThreads) total += (length_of(a, b) + kStep - 1) / kStep;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o);
  if (lane == 0) wsum[wave] = total;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kAWaves; ++w) total += wsum[w];
  total = wave_uniform64(total) * a.blocks;
  const int64_t per = range_steps(total);
  const int64_t start = blockIdx.x * per, end = min(total, start + per);
  int64_t before = 0;
  for (int b0 = 0; b0 < a.B; b0 += kAThreads) {
    const int b = b0 + tid;
    const int64_t n = b < a.B ? (length_of(a, b) + kStep - 1) / kStep : 0;
    int64_t incl = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t up = __shfl_up(incl, o);
      if (lane >= o) incl += up;
    }
    __syncthreads();
    if (lane == 63) wsum[wave] = incl;
    __syncthreads();
    int64_t sum = 0;
    for (int w = 0; w < kAWaves; ++w) {
      if (w == wave) incl += sum;
      sum += wsum[w];
    }
    incl += before;
    if (b < a.B) {
      const int64_t lo = (incl - n) * a.blocks;
      if (start >= lo && start < incl * a.blocks) {
        found[0] = b;
        found[1] = lo;
      }
      if (blockIdx.x == 0) {
        a.first[b] = incl - n;
        if (b == a.B - 1) a.first[a.B] = incl;
      }
    }
    before += sum;
  }
  __syncthreads();
  if (start >= total) return;
  int b = (int)wave_uniform64(found[0]);
  int64_t seq0 = wave_uniform64(found[1]);

  const int M = a.Sq * a.H;
  // lane offsets of the tile reads: rows of scores, transposed rows of values
  const int cb = latent_off<R>(col, grp), rb = tile_off<2 * kRope>(col, grp);
  // (this wave's value columns start at column block wd * kFrags)
  const int ct = (latent_off<R>(4 * grp + (col >> 2), (col & 3) >> 1) + ((col & 1) << 3)) ^ ((wd * kFrags & 7) << 5);
  for (int64_t at = start; at < end;) {
    int len = length_of(a, b);
    int n = (len + kStep - 1) / kStep;
    while (at >= seq0 + (int64_t)n * a.blocks) {   // the next sequence with steps
      seq0 += (int64_t)n * a.blocks;
      ++b;
      len = length_of(a, b);
      n = (len + kStep - 1) / kStep;
    }
    const int blk = (int)((at - seq0) / n), t0 = (int)((at - seq0) % n);
    const int t1 = (int)min((int64_t)n, t0 + (end - at));
    const bool whole = t0 == 0 && t1 == n;
    const int row = blk * kQRows + wq * 16 + col;
    const bool busy = blk * kQRows + wq * 16 < M;
    // rows that this lane's query sees
    const int limit = len - (a.Sq - 1 - min(row, M - 1) / a.H);

    bf8 qf[kSteps - kQLds];
    {
      const uint16_t* qp = a.q + ((int64_t)b * M + min(row, M - 1)) * (R + kRope) + 8 * grp;
#pragma unroll
      for (int s = 0; s < kSteps - kQLds; ++s) qf[s] = *reinterpret_cast<const bf8*>(qp + 32 * s);
#pragma unroll
      for (int s = 0; s < kQLds; ++s)
        qlds[wave][s][lane] = *reinterpret_cast<const bf8*>(qp + 32 * (kSteps - kQLds + s));
    }
    f4 o[kFrags];
#pragma unroll
    for (int d = 0; d < kFrags; ++d) o[d] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    float m = kNegInf, l = 0.0f;

    Stage<R, WT, FP8> stage;
    const int mine = wave * kRows + min(lane, kRows - 1);
    auto pos_of = [&](int t) { return t * kStep + mine; };
    // The copies of step t + 1 go to `next` while `cur` is worked on: the pointers are
    // declared not to alias, or the reads of `cur` would wait for them.
    auto step = [&](const LatentTile<R>* __restrict__ cur, LatentTile<R>* __restrict__ next, int t,
                    int& pg) __attribute__((always_inline)) {
      if constexpr (kCodes) {
        if (t + 1 < t1) convert_codes<R>(codes, next, wave, lane);
        if (t + 2 < t1) {
          copies_done();   // the codes are read before the next ones land on them
          copy_codes<R>(a, &codes, row_slot(a, pg, pos_of(t + 2), len), wave, lane);
          pg = page_of(a, b, pos_of(t + 3));
        }
      } else {
        if (t + 1 < t1) load_rows<R, WT, FP8>(a, stage, next, row_slot(a, pg, pos_of(t + 1), len), wave, lane);
        if (t + 2 < t1) pg = page_of(a, b, pos_of(t + 2));
      }
      const LatentTile<R>& tl = cur[wt];
      const int p0 = t * kStep + wt * kTok;   // position of the tile's first row
      if (busy && p0 < len) {
        f4 s[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
        // Row reads run kAhead products' worth ahead; the scheduling barriers keep them
        // there (left alone, every product waits for its own read).
        auto row_at = [&](int i, int f) {
          const uint8_t* k = i < R / 32 ? tl.c + f * 16 * 2 * R + (i >> 2) * 256 + (cb ^ ((i & 3) << 6))
                                        : tl.r + f * 16 * 2 * kRope + (rb ^ ((i - R / 32) << 6));
          return *reinterpret_cast<const bf8*>(k);
        };
        auto q_at = [&](int i) { return i < kSteps - kQLds ? qf[i] : qlds[wave][i - (kSteps - kQLds)][lane]; };
        bf8 kf[kAhead][2], qn[2] = {q_at(0), q_at(1)};
#pragma unroll
        for (int i = 0; i < kAhead; ++i) kf[i][0] = row_at(i, 0), kf[i][1] = row_at(i, 1);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          __builtin_amdgcn_sched_barrier(0);
          const bf8 q = qn[i % 2];
          s[0] = mfma16(kf[i % kAhead][0], q, s[0]);
          s[1] = mfma16(kf[i % kAhead][1], q, s[1]);
          if (i + 2 < kSteps) qn[i % 2] = q_at(i + 2);
          if (i + kAhead < kSteps) {
            kf[i % kAhead][0] = row_at(i + kAhead, 0);
            kf[i % kAhead][1] = row_at(i + kAhead, 1);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        const bool edge = p0 + kTok > len - (a.Sq - 1);
        float top = kNegInf;
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float x = s[f][r] * a.scale2;
            if (edge) x = p0 + 16 * f + 4 * grp + r < limit ? x : kNegInf;
            s[f][r] = x;
            top = fmaxf(top, x);
          }
        top = fmaxf(top, __shfl_xor(top, 16));
        top = half_max(top);
        // The running reference moves only when a score passes it by kSlack: the weights
        // stay below 2^kSlack, exact in FP32's and bf16's range, and the sums are seldom
        // rescaled. The first score of a row always sets it.
        const bool moved = top > m + kSlack || (m == kNegInf && top > kNegInf);
        if (__any(moved)) {
          const float to = moved ? top : m;
          const float shrink = to == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m - to);
          m = to;
          l *= shrink;
#pragma unroll
          for (int d = 0; d < kFrags; ++d) o[d] *= shrink;
        }
        const float base = m == kNegInf ? 0.0f : m;
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            s[f][r] = __builtin_amdgcn_exp2f(s[f][r] - base);
            l += s[f][r];
          }
        union { uint32_t u[4]; bf8 v; } p;
#pragma unroll
        for (int i = 0; i < 4; ++i) p.u[i] = pack_bf16x2(s[i / 2][2 * (i % 2)], s[i / 2][2 * (i % 2) + 1]);
        auto col_at = [&](int d) {
          // columns 16 (wd * kFrags + d)..: 4 rows a 16-lane group, of both 16-row halves
          typedef __attribute__((address_space(3))) bf4 lds_bf4;
          const uint8_t* v = tl.c + ((wd * kFrags >> 3) + (d >> 3)) * 256 + (ct ^ ((d & 7) << 5));
          const bf4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf4*)v);
          const bf4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf4*)(v + 16 * 2 * R));
          return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        };
        constexpr int kVAhead = kFrags < 6 ? kFrags : 6;
        bf8 vf[kVAhead];
#pragma unroll
        for (int d = 0; d < kVAhead; ++d) vf[d] = col_at(d);
#pragma unroll
        for (int d = 0; d < kFrags; ++d) {
          __builtin_amdgcn_sched_barrier(0);
          o[d] = mfma16(vf[d % kVAhead], p.v, o[d]);
          if (d + kVAhead < kFrags) vf[d % kVAhead] = col_at(d + kVAhead);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (FP8 && !kCodes) {
        if (t + 1 < t1) store_rows<R, WT>(stage, next, wave, lane);
      }
    };

    int pg = page_of(a, b, pos_of(t0));
    if constexpr (kCodes) {
      copy_codes<R>(a, &codes, row_slot(a, pg, pos_of(t0), len), wave, lane);
      pg = page_of(a, b, pos_of(t0 + 1));
      copies_done();
      convert_codes<R>(codes, tiles[t0 & 1], wave, lane);
      copies_done();
      if (t0 + 1 < t1) copy_codes<R>(a, &codes, row_slot(a, pg, pos_of(t0 + 1), len), wave, lane);
      pg = page_of(a, b, pos_of(t0 + 2));
    } else {
      load_rows<R, WT, FP8>(a, stage, tiles[t0 & 1], row_slot(a, pg, pos_of(t0), len), wave, lane);
      if constexpr (FP8) store_rows<R, WT>(stage, tiles[t0 & 1], wave, lane);
      pg = page_of(a, b, pos_of(t0 + 1));
    }
    for (int t = t0; t < t1; ++t) {
      copies_done_barrier();
      step(tiles[t & 1], tiles[(t + 1) & 1], t, pg);
    }
    l += __shfl_xor(l, 16);
    l = half_sum(l);
    if constexpr (WT == 2) {   // the second tile's waves hand their part to the first's
      copies_done_barrier();
      f4* x = reinterpret_cast<f4*>(tiles) + (wq * WD + wd) * kFrags * 64 + lane;
      float* ml = reinterpret_cast<float*>(reinterpret_cast<f4*>(tiles) + WQ * WD * kFrags * 64);
      static_assert(WQ * WD * (kFrags * 1024 + 512) <= (int)sizeof(tiles), "hand-over fits the tiles");
      if (wt == 1) {
#pragma unroll
        for (int d = 0; d < kFrags; ++d) x[d * 64] = o[d];
        ml[(wq * WD + wd) * 128 + lane] = m;
        ml[(wq * WD + wd) * 128 + 64 + lane] = l;
      }
      copies_done_barrier();
      if (wt == 0) {
        const float m1 = ml[(wq * WD + wd) * 128 + lane], l1 = ml[(wq * WD + wd) * 128 + 64 + lane];
        const float top = fmaxf(m, m1), base = top == kNegInf ? 0.0f : top;
        const float w0 = __builtin_amdgcn_exp2f(m - base), w1 = __builtin_amdgcn_exp2f(m1 - base);
        m = top;
        l = l * w0 + l1 * w1;
#pragma unroll
        for (int d = 0; d < kFrags; ++d) o[d] = o[d] * w0 + x[d * 64] * w1;
      }
    }
    if (busy && wt == 0) {
      if (whole) {
        if (row < M) {
          const float inv = l > 0.0f ? 1.0f / l : 0.0f;
          const int64_t to = ((int64_t)b * M + row) * R + wd * kCols + 4 * grp;
#pragma unroll
          for (int d = 0; d < kFrags; ++d)
            store4(a.out, to + 16 * d, a.out_bf16, o[d][0] * inv, o[d][1] * inv, o[d][2] * inv, o[d][3] * inv);
          if (grp == 0 && wd == 0)
            a.lse[(int64_t)b * M + row] = l > 0.0f ? (m + __builtin_amdgcn_logf(l)) * kLn2 : kNegInf;
        }
      } else {
        // lanes side by side: [wq][column block of 16][lane][4]
        float* p = a.part + ((int64_t)blockIdx.x * 2 + (at == start ? 0 : 1)) * part_floats(R, kQRows);
#pragma unroll
        for (int d = 0; d < kFrags; ++d)
          *reinterpret_cast<f4*>(p + ((wq * (R / 16) + wd * kFrags + d) * 64 + lane) * 4) = o[d];
        if (grp == 0 && wd == 0) {
          p[kQRows * R + wq * 16 + col] = m;
          p[kQRows * (R + 1) + wq * 16 + col] = l;
        }
      }
    }
    at += t1 - t0;
    copies_done_barrier();   // every wave is done with the tiles before the next block's
  }
}

// Joins the partial results of a block of query rows, or writes the empty result of a
// sequence without rows. A workgroup takes 16 query rows; a thread 4 columns at a time.
template <int R, int WQ>
__global__ __launch_bounds__(256) void absorbed_join_kernel(const AbsorbedArgs a) {
  constexpr int kQRows = 16 * WQ;
  const int unit = blockIdx.x;
  const int wq = unit % WQ, blk = unit / WQ % a.blocks, b = unit / WQ / a.blocks;
  const int lane = threadIdx.x & 63, col = lane & 15, grp = lane >> 4;
  const int M = a.Sq * a.H, row = blk * kQRows + wq * 16 + col;
  const int64_t n = a.first[b + 1] - a.first[b];
  const int64_t s0 = a.first[b] * a.blocks + blk * n, s1 = s0 + n;
  const int64_t per = range_steps(a.first[a.B] * a.blocks);
  const int64_t g0 = s0 / per, g1 = n > 0 ? (s1 - 1) / per : g0 - 1;
  if (g0 == g1 || row >= M) return;
  auto part = [&](int64_t g) { return a.part + (g * 2 + (s0 <= g * per ? 0 : 1)) * part_floats(R, kQRows); };
  float m = kNegInf;
  for (int64_t g = g0; g <= g1; ++g) m = fmaxf(m, part(g)[kQRows * R + wq * 16 + col]);
  const float base = m == kNegInf ? 0.0f : m;
  const int d = blockIdx.y * 4 + (threadIdx.x >> 6);
  float l = 0.0f;
  f4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int64_t g = g0; g <= g1; ++g) {
    const float* p = part(g);
    const float w = __builtin_amdgcn_exp2f(p[kQRows * R + wq * 16 + col] - base);
    l = fmaf(w, p[kQRows * (R + 1) + wq * 16 + col], l);
    const f4 v = *reinterpret_cast<const f4*>(p + ((wq * (R / 16) + d) * 64 + lane) * 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = fmaf(w, v[e], o[e]);
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  store4(a.out, ((int64_t)b * M + row) * R + 16 * d + 4 * grp, a.out_bf16, o[0] * inv, o[1] * inv, o[2] * inv,
         o[3] * inv);
  if (d == 0 && grp == 0)
    a.lse[(int64_t)b * M + row] = l > 0.0f ? (m + __builtin_amdgcn_logf(l)) * kLn2 : kNegInf;
}

// Query rows of a workgroup: as many 16-row groups as the query has, up to 8.
int query_rows(int M) { return M > 64 ? 128 : M > 32 ? 64 : M > 16 ? 32 : 16; }
size_t first_bytes(int64_t B) { return ((size_t)(B + 1) * 8 + 255) / 256 * 256; }

template <int R, int WQ, int WT, int WD>
void launch_absorbed(const AbsorbedArgs& a, bool fp8, hipStream_t s) {
  if (fp8) hipLaunchKernelGGL((absorbed_kernel<R, WQ, WT, WD, true>), dim3(kGroups), dim3(kAThreads), 0, s, a);
  else hipLaunchKernelGGL((absorbed_kernel<R, WQ, WT, WD, false>), dim3(kGroups), dim3(kAThreads), 0, s, a);
  hipLaunchKernelGGL((absorbed_join_kernel<R, WQ>), dim3((unsigned)(a.B * a.blocks * WQ), R / 64), dim3(256), 0, s, a);
}

template <int R>
void launch_rows(const AbsorbedArgs& a, bool fp8, hipStream_t s) {
  switch (query_rows(a.Sq * a.H)) {
    case 16: return launch_absorbed<R, 1, 2, 4>(a, fp8, s);
    case 32: return launch_absorbed<R, 2, 2, 2>(a, fp8, s);
    case 64: return launch_absorbed<R, 4, 1, 2>(a, fp8, s);
    default: return launch_absorbed<R, 8, 1, 1>(a, fp8, s);
  }
}

}  // namespace
}  // namespace moe

using namespace moe;

constexpr int kMaxSq = 64;
constexpr int64_t kMaxBatch = 65535;

extern "C" size_t moe_latent_attn_absorbed_workspace_bytes(const moe_latent_config* cfg, int64_t B, int32_t Sq) {
  if (check_latent(cfg) != MOE_OK || B < 0 || B > kMaxBatch || Sq < 1 || Sq > kMaxSq) return 0;
  return first_bytes(B) + (size_t)kGroups * 2 * part_floats(cfg->latent, query_rows(Sq * cfg->n_heads)) * 4;
}

extern "C" moe_status moe_latent_attn_absorbed(const moe_latent_config* cfg, int64_t B, int32_t Sq,
                                               const uint16_t* q, const void* cache, int64_t n_pages,
                                               int32_t page_size, const int32_t* page_table, int64_t max_pages,
                                               const int32_t* lengths, float scale, void* out, moe_dtype ot,
                                               float* lse, void* ws, size_t ws_bytes, void* stream) {
  const moe_status st = check_latent(cfg);
  if (st != MOE_OK) return st;
  if (Sq < 1 || Sq > kMaxSq || B < 0 || B > kMaxBatch || page_size < 1) return MOE_ERR_SHAPE;
  if (n_pages < 0 || n_pages > 0x7fffffff || n_pages * page_size > 0x7fffffff) return MOE_ERR_SHAPE;
  if (max_pages < 0 || max_pages > 0x7fffffff || max_pages * page_size > 0x7fffff00) return MOE_ERR_SHAPE;
  if (!good_scale(scale)) return MOE_ERR_SHAPE;
  if (ot != MOE_BF16 && ot != MOE_F32) return MOE_ERR_DTYPE;
  if (B == 0) return MOE_OK;
  if (!q || !lengths || !out || !lse || (max_pages > 0 && !page_table) || (n_pages > 0 && !cache)) return MOE_ERR_NULL;
  if (misaligned16(q) || misaligned16(cache) || misaligned16(out) || misaligned16(ws)) return MOE_ERR_UNSUPPORTED;
  if (!ws || ws_bytes < moe_latent_attn_absorbed_workspace_bytes(cfg, B, Sq)) return MOE_ERR_WORKSPACE;
  const int M = Sq * cfg->n_heads;
  const AbsorbedArgs a{q, static_cast<const uint8_t*>(cache), page_table, lengths, out, lse,
                       static_cast<int64_t*>(ws),
                       reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + first_bytes(B)), n_pages, max_pages,
                       (int)B, Sq, cfg->n_heads, page_size, (M + query_rows(M) - 1) / query_rows(M), scale * kLog2e,
                       ot == MOE_BF16};
  if ((int64_t)a.B * a.blocks * 8 > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  const bool fp8 = cfg->cache_kind == MOE_CACHE_FP8;
  if (cfg->latent == 512) launch_rows<512>(a, fp8, as_stream(stream));
  else launch_rows<256>(a, fp8, as_stream(stream));
  return launch_status();
}
