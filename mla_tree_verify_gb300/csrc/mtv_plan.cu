// Planner kernel of the MLA tree-verify path.
//
// Planner: one CTA turns kv_indptr / qo_indptr / mask_indptr into the balanced work
// plan that the split kernel walks, without any host round trip (the capture-safety
// requirement of "The Architecture of Capture Safety", section "The Design Emerges":
// fixed grid, sizes derived on the device, no .item()).
//
// Work plan (JobGeo in mtv_common.cuh).  A unit is one key tile of one job; the split
// CTAs form lane groups of `lanes` CTAs, and the lanes of a group walk the same units,
// each on its own column group (draft tokens) of the job, so that the draft tokens of a
// request read each key tile at about the same time and all but the first read hit L2.
// Each job also owns seg_cost empty units (the cost of a segment's start and end, about
// one tile).  Lane group g owns units [g C, (g + 1) C), where C is the larger of
// ceil(U / groups) and ceil(max_tiles / (NSPLIT - 2 lanes)), so that no column group is
// cut into more than NSPLIT = 64 partials ("The Architecture of Capture Safety" fixes
// NSPLIT at 64: section "The Design Emerges", first insight).  Each active lane of each job
// gets a lane-token index (cum_tok[b] + j lanes + r), and its piece in lane group g is
// written to partial slot tok + lanes g (SegMap in mtv_common.cuh).
//
// The merge of the partials runs at the end of the split kernel (merge_token() in
// mtv_common.cuh).
#include "mtv_common.cuh"
#include "mtv_q8.cuh"

namespace mtv {

// Inclusive block scans of two int64 and the maximum of a uint32 per thread (blockDim.x =
// kPlanThreads): v[i] becomes the sum of v[i] over threads 0..tid, total[i] the block's sum.
constexpr int kPlanThreads = 256;
struct PlanScan {
  int64_t sum[kPlanThreads / 32][2];
  uint32_t top[kPlanThreads / 32];
};

__device__ __forceinline__ void block_scan(PlanScan& sm, int64_t (&v)[2], int64_t (&total)[2], uint32_t& top) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, v[0], o), y = __shfl_up_sync(0xffffffffu, v[1], o);
    if (lane >= o) {
      v[0] += x;
      v[1] += y;
    }
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 31) {
    sm.sum[warp][0] = v[0];
    sm.sum[warp][1] = v[1];
    sm.top[warp] = top;
  }
  __syncthreads();
  total[0] = total[1] = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    const int64_t x = sm.sum[w][0], y = sm.sum[w][1];
    total[0] += x;
    total[1] += y;
    v[0] += w < warp ? x : 0;
    v[1] += w < warp ? y : 0;
    top = max(top, sm.top[w]);
  }
}

__device__ __forceinline__ void plan_body(const Problem& p, int32_t grid, int32_t tile) {
  __shared__ PlanScan s_scan;
  __shared__ int64_t s_cum[3][kPlanThreads + 1];   // with one pass: cum_units, cum_tok, cum_job
  __shared__ int32_t s_bad[32];      // requests whose mask block is inconsistent
  __shared__ int32_t s_nbad;
  // The split kernel may start its prologue now; it waits for this grid's results.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  if (tid == 0) {
    p.hdr->error_flags = 0u;
    p.hdr->merges_tmem = 0u;
    p.hdr->merges_ws = 0u;
    p.hdr->helps = 0u;
    p.hdr->helps_left = 0u;
    s_nbad = 0;
  }
  // One request per thread: its six indptr entries are loaded once (one round of
  // loads when bs <= blockDim; after an L2 flush each round is a trip to DRAM).
  struct Req { int64_t kv0, kv1, q0, q1, m0, m1; };
  auto load_req = [&](int64_t b) {
    Req r;
    r.kv0 = p.kv_indptr[b]; r.kv1 = p.kv_indptr[b + 1];
    r.q0 = p.qo_indptr[b]; r.q1 = p.qo_indptr[b + 1];
    r.m0 = p.mask_indptr[b]; r.m1 = p.mask_indptr[b + 1];
    return r;
  };
  const bool one_pass = p.bs <= (int32_t)blockDim.x;
  Req mine{0, 0, 0, 0, 0, 0};
  if (one_pass && tid < p.bs) mine = load_req(tid);
  for (int64_t i = tid; i < (int64_t)p.bs * p.max_q_per_req; i += blockDim.x) p.tok_done[i] = 0;
  for (int64_t i = tid; i < (int64_t)p.bs * p.max_q_per_req * kMergeFan; i += blockDim.x)
    p.grp_done[i] = 0;
  __syncthreads();

  // 1. indptr arrays must be in range and nondecreasing, else nothing is computed.
  auto indptr_bad = [&](const Req& r) {
    return r.kv0 < 0 || r.kv1 < r.kv0 || r.kv1 > p.num_kv_indices || r.q0 < 0 || r.q1 < r.q0 ||
           r.q1 > p.total_q || r.q1 - r.q0 > p.max_q_per_req;
  };
  int bad = 0;
  for (int64_t b = tid; b < p.bs; b += blockDim.x) bad |= indptr_bad(one_pass ? mine : load_req(b));
  bad = __syncthreads_or(bad);
  if (bad) {
    for (int64_t b = tid; b <= p.bs; b += blockDim.x) p.cum_units[b] = p.cum_tok[b] = p.cum_job[b] = 0;
    if (tid == 0) {
      atomicOr(&p.hdr->error_flags, kErrBadIndptr);
      p.hdr->total_units = 0;
      p.hdr->capacity = 1;
      p.hdr->max_tiles = 0;
      p.hdr->grid = grid;
      p.hdr->tile = tile;
      p.hdr->bs = p.bs;
      p.hdr->lanes = p.lanes;
      p.hdr->groups = grid / p.lanes;
    }
    return;
  }

  // 2. units, active lanes and jobs per request (a request whose mask block is
  //    inconsistent gets none), and their exclusive prefix sums, which stay in shared memory
  //    too when one pass does them.  Lanes and jobs are summed in one word: both stay below
  //    2^31 (at most T_b + 7 for a request with drafts, and total_q < 2^25).
  const GeoShift sh = geo_shift(p.group_tokens, p.lanes, tile);
  auto mask_bad = [&](const Req& r, int64_t T, int64_t L) {
    return r.m0 < 0 || r.m1 - r.m0 != T * L || r.m1 > p.mask_len;
  };
  int64_t units = 0, toks = 0, jobs = 0;   // sums so far
  uint32_t mt = 0;
  for (int64_t base = 0; base < p.bs; base += blockDim.x) {
    const int64_t b = base + tid;
    int64_t v[2] = {0, 0};   // units; lane tokens and jobs << 32
    uint32_t tiles = 0;
    if (b < p.bs) {
      const Req r = one_pass ? mine : load_req(b);
      const int64_t T = r.q1 - r.q0, L = (r.kv1 - r.kv0) + T;
      if (T > 0) {
        if (mask_bad(r, T, L)) {
          atomicOr(&p.hdr->error_flags, kErrBadMask);
          const int slot = atomicAdd(&s_nbad, 1);
          if (slot < 32) s_bad[slot] = (int32_t)b;
        } else {
          const JobGeo g = job_geo(L, (int32_t)T, sh, p.seg_cost);
          v[0] = req_units(g);
          v[1] = req_toks(g, p.lanes) | g.jobs << 32;
          tiles = (uint32_t)g.tiles;
        }
      }
    }
    const int64_t own[2] = {v[0], v[1]};
    int64_t total[2];
    block_scan(s_scan, v, total, tiles);
    mt = max(mt, tiles);
    if (b < p.bs) {
      const int64_t x = v[1] - own[1];
      const int64_t cu = units + v[0] - own[0], ct = toks + (x & 0xffffffff), cj = jobs + (x >> 32);
      p.cum_units[b] = cu;
      p.cum_tok[b] = ct;
      p.cum_job[b] = cj;
      if (one_pass) {
        s_cum[0][b] = cu;
        s_cum[1][b] = ct;
        s_cum[2][b] = cj;
      }
    }
    units += total[0];
    toks += total[1] & 0xffffffff;
    jobs += total[1] >> 32;
    __syncthreads();
  }
  // Rows of requests with an inconsistent mask block get out = 0, lse = -inf (no split
  // CTA visits them).
  {
    const int nbad = s_nbad;
    for (int64_t bi = 0; bi < p.bs; ++bi) {
      int64_t b;
      if (nbad <= 32) {
        if (bi >= nbad) break;
        b = s_bad[bi];
      } else {  // more than 32: test every request
        b = bi;
        const int64_t T = p.qo_indptr[b + 1] - p.qo_indptr[b];
        const int64_t L = ((int64_t)p.kv_indptr[b + 1] - p.kv_indptr[b]) + T;
        const int64_t m0 = p.mask_indptr[b], m1 = p.mask_indptr[b + 1];
        if (T == 0 || !(m0 < 0 || m1 - m0 != T * L || m1 > p.mask_len)) continue;
      }
      const int64_t q0 = p.qo_indptr[b], q1 = p.qo_indptr[b + 1];
      for (int64_t i = tid; i < (q1 - q0) * p.heads * (kDv / 8); i += blockDim.x)
        ((uint4*)(p.out + q0 * p.heads * kDv))[i] = make_uint4(0, 0, 0, 0);
      for (int64_t i = tid; i < (q1 - q0) * p.heads; i += blockDim.x)
        p.lse[q0 * p.heads + i] = -INFINITY;
    }
  }
  const int64_t groups = (int64_t)grid >> sh.lanes;
  // Units per lane group: an even share, at most 64 partials per column group, and at
  // least min(max_tiles, 3) + seg_cost, so that a small batch is not spread one tile per
  // CTA (every token would then need a merge that costs more than the tiles it saves).
  int64_t cap = max(udiv(units + groups - 1, groups),
                    udiv(mt + kNsplit - 2 * p.lanes - 1, kNsplit - 2 * p.lanes));
  cap = max(cap, min((int64_t)mt, (int64_t)3) + p.seg_cost);
  cap = max(cap, (int64_t)1);
  if (tid == 0) {
    p.cum_units[p.bs] = units;
    p.cum_tok[p.bs] = toks;
    p.cum_job[p.bs] = jobs;
    p.hdr->total_units = units;
    p.hdr->capacity = cap;
    p.hdr->max_tiles = mt;
    p.hdr->grid = grid;
    p.hdr->tile = tile;
    p.hdr->bs = p.bs;
    p.hdr->lanes = p.lanes;
    p.hdr->groups = (int32_t)groups;
  }
  // 3. the job records (the divisions by C happen here, so that the split kernel's walk has
  //    none), a thread each, and, from the last thread down, the first job of each lane group:
  //    that of its first unit, or 0 when it starts past the last unit and has no work.
  const int64_t* cum_u = one_pass ? s_cum[0] : p.cum_units;
  const int64_t* cum_t = one_pass ? s_cum[1] : p.cum_tok;
  const int64_t* cum_j = one_pass ? s_cum[2] : p.cum_job;
  for (int64_t i = tid; i < jobs; i += blockDim.x) {
    const int64_t b = unit_request(cum_j, p.bs, i), j = i - cum_j[b];
    const Req r = load_req(b);
    const int64_t T = r.q1 - r.q0, P = r.kv1 - r.kv0;
    const JobGeo g = job_geo(P + T, (int32_t)T, sh, p.seg_cost);
    int32_t nt, k;
    int64_t sl;
    job_shape(g, j, p.lanes, nt, k, sl);
    JobRec rec;
    rec.js = cum_u[b] + j * g.hf;
    rec.m_base = r.m0;
    rec.tok0 = (int32_t)(cum_t[b] + j * p.lanes);
    rec.b = (int32_t)b;
    rec.kv_base = (int32_t)r.kv0;
    rec.P = (int32_t)P;
    rec.T = (int32_t)T;
    rec.q_base = (int32_t)r.q0;
    rec.cg0 = (int32_t)(j * p.lanes);
    rec.tiles = (int32_t)g.tiles;
    rec.sl = (int32_t)sl;
    rec.nt = nt;
    rec.k = k;
    int32_t nseg;
    const SegMap m = seg_map(0, 0, p.lanes, 0, rec.js, g.tiles, nt, sl, cap, nseg);
    rec.g_lo = (int32_t)m.g_lo;
    rec.n_full = m.n_full;
    rec.ns = m.ns;
    rec.nseg = nseg;
    rec.pad = 0;
    p.jobs[i] = rec;
  }
  for (int64_t gi = blockDim.x - 1 - tid; gi < groups; gi += blockDim.x) {
    const int64_t u = gi * cap;
    int64_t job = 0;
    if (u < units) {
      const int64_t b = unit_request(cum_u, p.bs, u);
      const Req r = load_req(b);
      const JobGeo g = job_geo(r.kv1 - r.kv0 + r.q1 - r.q0, (int32_t)(r.q1 - r.q0), sh, p.seg_cost);
      job = cum_j[b] + min(udiv(u - cum_u[b], g.hf), g.jobs - 1);
    }
    p.grp_job[gi] = (int32_t)job;
  }
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(Problem p, int32_t grid, int32_t tile) {
  plan_body(p, grid, tile);
}

void launch_plan(const Problem& p, int grid, int tile, cudaStream_t stream) {
  plan_kernel<<<1, kPlanThreads, 0, stream>>>(p, grid, tile);
}

// ---- the 8-bit cache's queries ----
// One warp per (token, head) row: x = q 2^(7 - e), e the exponent of the row's largest |q|, as
// hi = e4m3(x) and lo = e4m3(x - hi) (mtv_split_q8.cu), and the factor sm_scale log2(e) 2^(e-7)
// that the scores are multiplied by.  bf16 to f16 is exact here (|x| < 256, and what f16 cannot
// hold lies below 2^-24, far under e4m3's smallest step 2^-9).  A row with a NaN or an infinity
// gets zeros and a NaN factor.  Runs beside the planner, in the same launch.
__device__ __forceinline__ void split_q_row(const Problem& p, int64_t src_row, int64_t row) {
  const int lane = threadIdx.x & 31;
  const uint4* src = (const uint4*)(p.q + src_row * kDqk);   // 72 granules of 8 values
  uint4 w[3];
  w[0] = src[lane];
  w[1] = src[lane + 32];
  w[2] = lane < 8 ? src[lane + 64] : make_uint4(0, 0, 0, 0);
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const uint32_t v[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, max(v[i] << 16 & 0x7fffffffu, v[i] & 0x7fff0000u));
  }
  top = __reduce_max_sync(0xffffffffu, top);
  const bool bad = top >= 0x7f800000u;
  const int e = top == 0u || bad ? 7 : max((int)(top >> 23) - 127, -118);   // 2^(7-e) fits fp32
  const float up = __int_as_float((7 - e + 127) << 23);
  uint8_t* hi = p.q_split + row * q8::kRow;
  uint8_t* lo = hi + p.q_rows * q8::kRow;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (k == 2 && lane >= 8) break;
    const uint32_t v[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 x = __floats2half2_rn(__uint_as_float(v[i] << 16) * up,
                                          __uint_as_float(v[i] & 0xffff0000u) * up);
      h[i] = bad ? 0u : q8::pack2(*(const uint32_t*)&x);
      const uint32_t back = q8::unpack2(h[i]);
      const __half2 rest = __hsub2(x, *(const __half2*)&back);
      l[i] = bad ? 0u : q8::pack2(*(const uint32_t*)&rest);
    }
    const int g = lane + 32 * k;
    *(uint2*)(hi + 8 * g) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    *(uint2*)(lo + 8 * g) = make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
  }
  if (lane == 0)
    p.q_factor[row] = bad ? __int_as_float(0x7fc00000)
                          : p.sm_scale * 1.4426950408889634f * __int_as_float((e - 7 + 127) << 23);
}

// CTA 0 plans; the others split the queries of rows [qo_indptr[0], qo_indptr[bs]).
__global__ void __launch_bounds__(kPlanThreads, 4) plan_q8_kernel(Problem p, int32_t grid, int32_t tile) {
  if (blockIdx.x == 0) {
    plan_body(p, grid, tile);
    return;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t q0 = p.qo_indptr[0], q1 = p.qo_indptr[p.bs];
  if (q0 < 0 || q1 < q0 || q1 > p.total_q || (q1 - q0) * p.heads > p.q_rows) return;  // planner flags it
  const int64_t n = (q1 - q0) * p.heads, step = (int64_t)(gridDim.x - 1) * (blockDim.x / 32);
  for (int64_t r = (int64_t)(blockIdx.x - 1) * (blockDim.x / 32) + (threadIdx.x >> 5); r < n; r += step)
    split_q_row(p, q0 * p.heads + r, r);
}

void launch_plan_q8(const Problem& p, int grid, int tile, cudaStream_t stream) {
  // a row a warp up to 8 CTAs an SM, then rows in turn
  const int64_t rows = p.total_q * p.heads < p.q_rows ? p.total_q * p.heads : p.q_rows;
  const int64_t ctas = (rows + 7) / 8 < (int64_t)8 * grid ? (rows + 7) / 8 : (int64_t)8 * grid;
  plan_q8_kernel<<<(unsigned)(1 + ctas), kPlanThreads, 0, stream>>>(p, grid, tile);
}

}  // namespace mtv
