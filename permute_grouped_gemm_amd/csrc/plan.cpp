// Host-side validation and workspace planning (shapes only; no HIP calls).
//
// Validation follows the constraints table of the MoeInitRoutingGroupedMatmulGrad
// design page (§1.2) and its infershape checks (§2.3.3).  The schedule splits
// the expert-ordered list of m-tiles into chunks whose fp32 output rows fit a
// ring of bounded size, so the workspace does not grow with M·K.
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <cmath>

#include "pgg_internal.h"

namespace pgg {

namespace {

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Bound on the fp32 ring (bytes): 1 GiB, a fixed amount whatever M (0.35 %
// of an MI355X's 288 GB).  Measured against 256 and 512 MiB with the panel
// choice below: the large fp16 call (M 110592, K 7168, N 2048) took 3.92
// against 4.34 and 4.07 ms, fewer chunks per panel meaning fewer
// read-modify-writes of d_x.  PGG_RING_MB lowers it for tuning; a fixed
// setting gives fixed results.  At most 1 GiB: ring offsets stay below 2^30
// bytes.
size_t ring_budget() {
  constexpr long kMaxMb = 1024;
  const char* e = getenv("PGG_RING_MB");
  if (e) {
    long mb = strtol(e, nullptr, 10);
    if (mb > 0) return static_cast<size_t>(std::min<long>(mb, kMaxMb)) << 20;
  }
  return static_cast<size_t>(kMaxMb) << 20;
}

struct TileShape { int bm, bn; };

// Columns per panel when K is cut into n panels: whole tiles of bn columns.
int64_t panel_width(int64_t K, int n, int bn) {
  const int64_t w = (K + n - 1) / n;
  return std::min<int64_t>(K, (w + bn - 1) / bn * bn);
}

// m-tiles per chunk when a ring row holds `cols` fp32 columns.
int64_t tiles_per_chunk(int bm, int64_t cols, size_t budget, int64_t max_tiles) {
  const size_t per_tile = size_t(bm) * size_t(cols) * sizeof(float);
  const int64_t tc = static_cast<int64_t>(budget / per_tile);
  return std::max<int64_t>(1, std::min<int64_t>(tc, max_tiles));
}

// Panel count.  PGG_PANEL_COLS fixes the panel width (tuning; a fixed
// setting gives fixed results).  Otherwise a time estimate picks it, with
// rates measured on MI355X at the large fp16, large fp32 and mid bf16 shapes:
//  - the consumer reads every ring row once.  With C chunks per panel, each
//    of a token's topK rows in any chunk alike, the token's rows fall in
//    E = C (1 - (1 - 1/C)^topK) distinct chunks and its d_x row is read and
//    written 2E - 1 times (once when C = 1); it moves these bytes at about
//    6.4-6.8 TB/s with up to 3 chunks per panel, about 5 TB/s with 4 (the
//    chunk consumer) and about 5 TB/s by ring row (more chunks);
//  - every panel past the first reads d_y again: about 15 TB/s of extra
//    reads for the 16-bit producers, which hide most of it behind the
//    multiply, and 4.7 TB/s for the fp32 producer;
//  - the large-tile producer runs one 256 x 256 tile per compute unit at a
//    time, so a launch of T tiles takes ceil(T / 256) rounds of about
//    21 us + 0.022 us x N each for 16-bit inputs (measured at N = 2048 and
//    4096), and about 16 times that per N for fp32 (the MFMA rate).  The
//    true m-tile count is known only on the device; rounds are counted at
//    its expectation under routing that is uniform over the experts
//    (expected_tiles), cut into chunks of the plan's size (which the bound
//    sets).  The bound (M / 256 plus one partial tile per expert)
//    overstates a launch by up to G / 2 m-tiles, which at 64 experts of
//    about 512 rows (K 7168, N 2048) made 7 panels of one chunk look as fast
//    as 2 panels of three, against 1.52 and 1.38 ms measured.
// The weight-streaming producer keeps one panel.
// Rounds of the large-tile producer over all panels of width w with chunks
// of tc m-tiles, for `tiles` m-tiles.
int64_t producer_rounds(const Plan& q, int64_t w, int64_t tc, int64_t tiles) {
  constexpr int64_t kCUs = 256;
  int64_t rounds = 0;
  for (int64_t k0 = 0; k0 < q.K; k0 += w) {
    const int64_t ct = (std::min<int64_t>(w, q.K - k0) + q.bn - 1) / q.bn;
    for (int64_t left = tiles; left > 0; left -= tc)
      rounds += (std::min<int64_t>(left, tc) * ct + kCUs - 1) / kCUs;
  }
  return rounds;
}

// Expected m-tiles of bm rows per expert when each token's topK experts are
// distinct and uniform: an expert's row count is then Binomial(batch, topK /
// G), and E[ceil(c / bm)] = sum_j P(c > j bm), taken from the normal
// approximation with continuity correction.  Terms more than 8 standard
// deviations below the mean are 1 and are counted without the loop, so the
// loop runs over at most 16 sd / bm + 2 terms.
double expected_tiles_per_expert(const Plan& q, int bm) {
  const double p = std::min(1.0, double(q.topk) / double(q.G));
  const double mu = double(q.batch) * p;
  const double sd = std::sqrt(double(q.batch) * p * (1.0 - p));
  const int64_t j0 = static_cast<int64_t>(std::max(0.0, mu - 8.0 * sd - 1.0) / bm);
  double per_expert = double(j0);
  for (int64_t j = j0; double(j) * bm < mu + 8.0 * sd + 1.0; ++j) {
    const double x = double(j) * bm;
    per_expert += sd > 0.0 ? 0.5 * std::erfc((x + 0.5 - mu) / (sd * std::sqrt(2.0))) : (mu > x ? 1.0 : 0.0);
  }
  return per_expert;
}

// The same over all experts, clamped to [ceil(M / bm), max_tiles].
int64_t expected_tiles(const Plan& q, int64_t max_tiles) {
  const int64_t lo = (q.M + q.bm - 1) / q.bm;
  const int64_t est = static_cast<int64_t>(std::ceil(expected_tiles_per_expert(q, q.bm) * double(q.G)));
  return std::max<int64_t>(lo, std::min<int64_t>(est, max_tiles));
}

// Producer family, and for the fp32 tiles their height.  Measured on MI355X
// with uniform routing (K x N of 7168 x 4096, 7168 x 2048 and 2048 x 1408;
// 16, 60 and 64 experts):
//  - 16-bit: the weight sweep reads every expert's weights once per 32-row
//    m-tile, the 256 x 256 tiles once per 256 rows.  The sweep is faster up
//    to 24 rows per expert (197 against 236 us, 405 against 456 us) and the
//    tiles from 32 (240 against 253 us, 473 against 534 us, 112 against 140
//    us), so the sweep takes M <= 28 G.
//  - fp32 up to 32 rows per expert: the weight sweep (fp32 MFMAs on the same
//    staged chunks), 359 against 1057 us for the 128 x 128 tile at 8 rows
//    per expert (16 experts, 7168 x 4096); at 32 it ties with the 64 x 128
//    tile (606 against about 600 us) and at 48 it loses (921 against 598).
//  - fp32 above that: the tiles are bound by the fp32 MFMAs, which also
//    multiply the padding rows of each expert's last m-tile.  The tile with
//    the least expected padded rows at its relative rate is taken: 0.73 for
//    64 x 128, 0.78 for 128 x 128 and 0.85 for the direct-to-LDS 256 x 256,
//    fitted to the measured choices: 64 rows at 48-64, 128-256 rows per
//    expert (598 against 1081 us at 48, 1469 against 1631 at 128), 128 rows
//    at 96 (1100 against 1175 us), 256 rows at 192 and 1024 and at the large
//    fp32 shape (1.95 against 2.04 ms, 16.05 against 16.51 ms, 25.4 against
//    27.4 ms).
struct Family {
  int32_t regime;
  int32_t bm;   // fp32 tile rows (kF32 only)
};

Family choose_family(const Plan& q) {
  if (q.dtype != PGG_F32) return {q.M <= 28 * q.G ? kStream : kLarge, 0};
  const double c64 = expected_tiles_per_expert(q, 64) * 64.0 / 0.73;
  const double c128 = expected_tiles_per_expert(q, 128) * 128.0 / 0.78;
  const double c256 = expected_tiles_per_expert(q, 256) * 256.0 / 0.85;
  const int32_t bm = c64 <= c128 ? 64 : 128;
  if (q.M <= 32 * q.G) return {kStream, bm};
  if (c256 < std::min(c64, c128)) return {kLarge, bm};
  return {kF32, bm};
}

int choose_panels(const Plan& q, size_t budget, int64_t max_tiles) {
  // the weight sweep stores whole K-column ring rows: one panel, whatever the override
  if (q.regime == kStream) return 1;
  const int64_t max_panels = (q.K + q.bn - 1) / q.bn;
  if (const char* e = getenv("PGG_PANEL_COLS")) {
    const long c = strtol(e, nullptr, 10);
    if (c > 0) {
      const int64_t w = std::min<int64_t>(q.K, (c + q.bn - 1) / q.bn * q.bn);
      return static_cast<int>((q.K + w - 1) / w);
    }
  }
  constexpr double kConsumeRate = 6.7, kManyChunkRate = 5.0;
  constexpr int64_t kFastChunks = 3;
  const double reread_rate = q.dtype == PGG_F32 ? 4.7 : 15.0;
  const double elem = q.dtype == PGG_F32 ? 4.0 : 2.0;
  const double dy_bytes = double(q.M) * double(q.N) * elem;
  const double ring_bytes = double(q.M) * double(q.K) * 4.0;
  const double dx_bytes = double(q.batch) * double(q.K) * 4.0;
  // one round of 256 x 256 tiles, in ps (fp32: the MFMA rate is 16 times lower)
  const double round_ps = 21.0e6 + (q.dtype == PGG_F32 ? 230.0e3 : 22.0e3) * double(q.N);
  const int64_t est_tiles = expected_tiles(q, max_tiles);
  int best = 1;
  double best_time = 0.0;
  int64_t last_width = -1;
  for (int64_t n = 1; n <= std::min<int64_t>(max_panels, 64); ++n) {
    const int64_t w = panel_width(q.K, static_cast<int>(n), q.bn);
    if (w == last_width) continue;   // same width as a smaller count
    last_width = w;
    const int64_t panels = (q.K + w - 1) / w;
    const int64_t tc = tiles_per_chunk(q.bm, w, budget, max_tiles);
    const int64_t chunks = (max_tiles + tc - 1) / tc;
    const double c = double(chunks);
    const double e = c * (1.0 - std::pow(1.0 - 1.0 / c, double(q.topk)));
    double t = (ring_bytes + dx_bytes * (2.0 * e - 1.0)) /
               (chunks <= kFastChunks ? kConsumeRate : kManyChunkRate);
    t += double(panels - 1) * dy_bytes / reread_rate;
    if (q.regime == kLarge) t += double(producer_rounds(q, w, tc, est_tiles)) * round_ps;
    if (n == 1 || t < best_time) {
      best = static_cast<int>(panels);
      best_time = t;
    }
  }
  return best;
}

// Output tile per regime: large-M MFMA tiles (every input type); for few rows
// per expert, m-tiles of 32 rows crossed with units of 16 weight rows that a
// persistent grid streams in address order; for fp32 in between, tiles 128
// wide and 64 or 128 rows high (the height chosen with the family).
TileShape tile_shape(int32_t regime) {
  switch (regime) {
    case kLarge: return {256, 256};
    case kStream: return {32, 16};
    default: return {128, 128};
  }
}

}  // namespace

namespace {

pgg_status plan_with_budget(const pgg_moe_dx_desc* d, size_t budget, Plan* p) {
  if (!d || !p) return PGG_ERR_INVALID_ARG;
  const int64_t M = d->grad_y_rows, N = d->grad_y_cols;
  const int64_t G = d->weight_groups, K = d->weight_rows;
  if (d->reserved != 0) return PGG_ERR_INVALID_ARG;
  if (d->topk <= 0 || d->batch <= 0) return PGG_ERR_INVALID_ARG;
  if (d->row_idx_type != 0 && d->row_idx_type != 1) return PGG_ERR_INVALID_ARG;
  if (d->grad_y_dtype != d->weight_dtype) return PGG_ERR_INVALID_ARG;
  if (d->grad_y_dtype < PGG_F32 || d->grad_y_dtype > PGG_BF16) return PGG_ERR_INVALID_ARG;
  if (N != d->weight_cols) return PGG_ERR_INVALID_ARG;
  if (d->group_list_len != G) return PGG_ERR_INVALID_ARG;
  if (G <= 0 || K <= 0 || N <= 0 || M <= 0) return PGG_ERR_INVALID_ARG;
  if (d->topk > INT64_MAX / d->batch) return PGG_ERR_INVALID_ARG;
  if (M != d->batch * d->topk) return PGG_ERR_INVALID_ARG;
  const int64_t L = d->idx_len;
  if (L < d->batch || L > d->batch * d->topk || L < M) return PGG_ERR_INVALID_ARG;
  // Row indices are kept as int32 on the device; the page limits M to 2^31.
  if (M >= (int64_t(1) << 31) - 1) return PGG_ERR_UNSUPPORTED;
  if (G >= (int64_t(1) << 30) || K >= (int64_t(1) << 31) || N >= (int64_t(1) << 31))
    return PGG_ERR_UNSUPPORTED;
  // the consumer addresses a d_x row (4K bytes) through a 32-bit range
  if (K >= (int64_t(1) << 29)) return PGG_ERR_UNSUPPORTED;

  Plan q{};
  q.n_panels = 1;
  q.M = M; q.N = N; q.G = G; q.K = K; q.batch = d->batch; q.topk = d->topk;
  q.row_idx_type = d->row_idx_type;
  q.panel_cols = q.K;
  q.dtype = d->grad_y_dtype;
  // few rows per expert: the weight sweep, or for fp32 between the sweep and
  // the large tile the 64 x 128 or 128 x 128 tile
  const Family fam = choose_family(q);
  q.regime = fam.regime;
  // Non-temporal weight loads in the large tiles pay when each expert has
  // about one 256-row m-tile, so no other tile reads its slabs (measured:
  // 6-9 % faster at 64-128 rows per expert, 4-7 % slower at the large and mid
  // shapes, where every slab serves several m-tiles through L2).
  q.stream_weights = expected_tiles_per_expert(q, 256) <= 1.25;
  // PGG_REGIME=large, =few or =sweep fixes the producer family (tuning)
  if (const char* e = getenv("PGG_REGIME")) {
    if (!strcmp(e, "large")) q.regime = kLarge;
    else if (!strcmp(e, "few")) q.regime = q.dtype == PGG_F32 ? kF32 : kStream;
    else if (!strcmp(e, "sweep")) q.regime = kStream;
  }
  const TileShape ts = tile_shape(q.regime);
  q.bm = q.regime == kF32 ? fam.bm : ts.bm;
  q.bn = ts.bn;
  // 16-bit tiles 128 rows high (three LDS stages) when each expert has about
  // one such m-tile: measured 6-16 % faster than the 256-row tiles at 32-96
  // rows per expert, slower from 128 (two m-tiles for half the experts).
  if (q.regime == kLarge && q.dtype != PGG_F32 && q.stream_weights &&
      expected_tiles_per_expert(q, 128) <= 1.2)
    q.bm = 128;
  const int64_t max_tiles = (M + q.bm - 1) / q.bm + G;
  if (max_tiles >= (int64_t(1) << 31)) return PGG_ERR_UNSUPPORTED;
  q.max_tiles = static_cast<int32_t>(max_tiles);
  // Column panels: the output columns are cut into panels of panel_cols
  // (a multiple of the tile width), and every panel runs the whole chunk
  // sequence over the rows.  A ring row then holds one panel's columns, so a
  // chunk holds K / panel_cols times more rows: fewer chunks touch each token,
  // and the consumer re-reads and re-writes fewer d_x rows, at the price of
  // reading d_y once per panel.
  const int n_panels = choose_panels(q, budget, max_tiles);
  q.n_panels = n_panels;
  q.panel_cols = panel_width(K, n_panels, q.bn);
  int64_t tc = tiles_per_chunk(q.bm, q.panel_cols, budget, max_tiles);
  // keep the consumer grid (ring rows x column blocks of 256) well inside 2^31 work-items
  const int64_t col_blocks_worst = (int64_t(q.panel_cols) + 255) / 256;
  while (tc > 1 && tc * q.bm * col_blocks_worst >= (int64_t(1) << 23)) tc /= 2;
  if (int64_t(q.bm) * col_blocks_worst >= (int64_t(1) << 23)) return PGG_ERR_UNSUPPORTED;
  q.tc = static_cast<int32_t>(tc);
  q.max_chunks = static_cast<int32_t>((max_tiles + tc - 1) / tc);
  // a chunk's rows are at most its tiles' capacity and at most M; producers store
  // only the rows their tiles hold, at (row - first row of the chunk)
  q.ring_rows = static_cast<int32_t>(std::min<int64_t>(int64_t(q.tc) * q.bm, M));
  // column tiles of one panel (the last panel may use fewer)
  q.n_col_tiles = static_cast<int32_t>((q.panel_cols + q.bn - 1) / q.bn);
  q.fused_prep = M <= 16384;
  q.ksplit = 1;
  q.kspan = static_cast<int32_t>(N);

  size_t off = 0;
  q.off_header = off;   off = align_up(off + sizeof(WsHeader), kRegionAlign);
  q.off_offsets = off;  off = align_up(off + sizeof(int64_t) * size_t(G + 1), kRegionAlign);
  q.off_tiles = off;    off = align_up(off + sizeof(MTile) * size_t(q.max_tiles), kRegionAlign);
  q.off_chunks = off;   off = align_up(off + sizeof(int32_t) * size_t(q.max_chunks + 1), kRegionAlign);
  q.off_inv = off;      off = align_up(off + sizeof(int32_t) * size_t(M), kRegionAlign);
  q.off_ori = off;      off = align_up(off + sizeof(int32_t) * size_t(M), kRegionAlign);
  q.table_bytes = off;
  q.off_ring = off;
  q.ring_bytes = size_t(q.ring_rows) * size_t(q.panel_cols) * sizeof(float);
  off = align_up(off + q.ring_bytes, kRegionAlign);
  q.total = off;
  *p = q;
  return PGG_OK;
}

}  // namespace

pgg_status make_plan(const pgg_moe_dx_desc* d, Plan* p) {
  return plan_with_budget(d, ring_budget(), p);
}

pgg_status make_plan_within(const pgg_moe_dx_desc* d, size_t max_total, Plan* p) {
  Plan q;
  pgg_status st = plan_with_budget(d, ring_budget(), &q);
  if (st != PGG_OK) return st;
  // the tables' size with the largest possible chunk table (one chunk per m-tile)
  const size_t tables = q.table_bytes +
                        align_up(sizeof(int32_t) * size_t(q.max_tiles + 1), kRegionAlign) + kRegionAlign;
  if (max_total <= tables) return PGG_ERR_WORKSPACE_TOO_SMALL;
  st = plan_with_budget(d, std::min(ring_budget(), max_total - tables), &q);
  if (st != PGG_OK) return st;
  if (q.total > max_total) return PGG_ERR_WORKSPACE_TOO_SMALL;
  *p = q;
  return PGG_OK;
}

pgg_status make_fwd_plan(const pgg_moe_fwd_desc* d, Plan* p) {
  if (!d || !p) return PGG_ERR_INVALID_ARG;
  const int64_t batch = d->x_rows, K = d->x_cols;
  const int64_t G = d->weight_groups, N = d->weight_cols;
  if (d->reserved != 0) return PGG_ERR_INVALID_ARG;
  if (d->topk <= 0 || d->batch <= 0 || batch != d->batch) return PGG_ERR_INVALID_ARG;
  if (d->row_idx_type != 0 && d->row_idx_type != 1) return PGG_ERR_INVALID_ARG;
  if (d->x_dtype != d->weight_dtype) return PGG_ERR_INVALID_ARG;
  if (d->x_dtype < PGG_F32 || d->x_dtype > PGG_BF16) return PGG_ERR_INVALID_ARG;
  if (K != d->weight_rows) return PGG_ERR_INVALID_ARG;
  if (d->group_list_len != G) return PGG_ERR_INVALID_ARG;
  if (G <= 0 || K <= 0 || N <= 0) return PGG_ERR_INVALID_ARG;
  if (d->topk > INT64_MAX / d->batch) return PGG_ERR_INVALID_ARG;
  const int64_t M = d->batch * d->topk;
  if (d->idx_len != M) return PGG_ERR_INVALID_ARG;
  if (M >= (int64_t(1) << 31) - 1) return PGG_ERR_UNSUPPORTED;
  if (G >= (int64_t(1) << 30) || K >= (int64_t(1) << 31) || N >= (int64_t(1) << 31))
    return PGG_ERR_UNSUPPORTED;

  Plan q{};
  q.n_panels = 1;
  q.M = M; q.N = K; q.G = G; q.K = N; q.batch = d->batch; q.topk = d->topk;
  q.row_idx_type = d->row_idx_type;
  q.panel_cols = q.K;
  q.dtype = d->x_dtype;
  if (q.dtype == PGG_F32) {
    q.regime = kF32;
    q.bm = 128; q.bn = 128;
  } else if (M <= 64 * G) {
    q.regime = kStream;   // few rows per expert: 32-row m-tiles
    q.bm = 32; q.bn = 256;
  } else {
    q.regime = kLarge;
    q.bm = 256; q.bn = 256;
  }
  const int64_t max_tiles = (M + q.bm - 1) / q.bm + G;
  const int64_t col_tiles = (N + q.bn - 1) / q.bn;
  // the launch grid covers max_tiles x col_tiles workgroups
  if (max_tiles * col_tiles >= (int64_t(1) << 31) - 8 * 32) return PGG_ERR_UNSUPPORTED;
  q.max_tiles = static_cast<int32_t>(max_tiles);
  q.tc = q.max_tiles;
  q.max_chunks = 1;
  q.ring_rows = 0;
  q.n_col_tiles = static_cast<int32_t>(col_tiles);
  q.fused_prep = M <= 16384;
  // Few rows per expert: each tile streams its expert's weight columns over
  // the whole reduction.  When the tiles alone would leave the GPU short of
  // workgroups (at most max_tiles x col_tiles have work), the reduction is
  // split so that up to about 512 workgroups stream at once: one per resident
  // slot (two per compute unit).  More would run as a second, partly empty
  // wave (at the decode shape 2 splits took 133 us, 3 took 146 us, 4 took
  // 139 us).  Each split writes an fp32 partial of y and a reduction kernel
  // adds them in split order.
  q.ksplit = 1;
  q.kspan = static_cast<int32_t>(K);
  if (q.regime == kStream) {
    constexpr int64_t kStage = 64, kMinSpan = 512, kTarget = 512;
    const int64_t units = max_tiles * col_tiles;
    int64_t split = (kTarget + units - 1) / units;
    split = std::min<int64_t>(split, std::max<int64_t>(1, K / kMinSpan));
    split = std::max<int64_t>(1, std::min<int64_t>(split, 8));
    int64_t span = (K + split - 1) / split;
    span = (span + kStage - 1) / kStage * kStage;
    split = (K + span - 1) / span;
    q.ksplit = static_cast<int32_t>(split);
    q.kspan = static_cast<int32_t>(span);
  }

  size_t off = 0;
  q.off_header = off;   off = align_up(off + sizeof(WsHeader), kRegionAlign);
  q.off_offsets = off;  off = align_up(off + sizeof(int64_t) * size_t(G + 1), kRegionAlign);
  q.off_tiles = off;    off = align_up(off + sizeof(MTile) * size_t(q.max_tiles), kRegionAlign);
  q.off_chunks = off;   off = align_up(off + sizeof(int32_t) * size_t(q.max_chunks + 1), kRegionAlign);
  q.off_inv = off;      off = align_up(off + sizeof(int32_t) * size_t(M), kRegionAlign);
  q.off_ori = off;      off = align_up(off + sizeof(int32_t) * size_t(M), kRegionAlign);
  q.table_bytes = off;
  q.off_ring = off;
  q.ring_bytes = q.ksplit > 1 ? size_t(q.ksplit) * size_t(M) * size_t(N) * sizeof(float) : 0;
  q.ring_rows = q.ksplit > 1 ? static_cast<int32_t>(q.ksplit * M) : 0;
  off = align_up(off + q.ring_bytes, kRegionAlign);
  q.total = off;
  *p = q;
  return PGG_OK;
}

pgg_status make_routing_plan(const pgg_moe_routing_desc* d, RoutePlan* p) {
  if (!d || !p) return PGG_ERR_INVALID_ARG;
  if (d->reserved != 0 || d->batch <= 0 || d->topk <= 0 || d->experts <= 0 || d->x_cols < 0)
    return PGG_ERR_INVALID_ARG;
  if (d->x_cols > 0 && (d->x_dtype < PGG_F32 || d->x_dtype > PGG_BF16)) return PGG_ERR_INVALID_ARG;
  if (d->topk > INT64_MAX / d->batch) return PGG_ERR_INVALID_ARG;
  const int64_t M = d->batch * d->topk;
  constexpr int64_t kBlockPos = 1024;
  if (M >= (int64_t(1) << 31) - 1 || d->experts > 8192) return PGG_ERR_UNSUPPORTED;
  // the gather splits a row into pieces of at least 4 KiB along a grid
  // dimension of at most 65535
  if (d->x_cols >= (int64_t(1) << 25)) return PGG_ERR_UNSUPPORTED;
  const int64_t nblocks = (M + kBlockPos - 1) / kBlockPos;
  if (nblocks * d->experts >= (int64_t(1) << 28)) return PGG_ERR_UNSUPPORTED;
  RoutePlan q{};
  q.M = M;
  q.G = d->experts;
  q.topk = d->topk;
  q.K = d->x_cols;
  q.dtype = d->x_dtype;
  q.nblocks = static_cast<int32_t>(nblocks);
  size_t off = 0;
  q.off_header = off;  off = align_up(off + sizeof(WsHeader), kRegionAlign);
  q.off_table = off;   off = align_up(off + sizeof(int32_t) * size_t(nblocks * q.G), kRegionAlign);
  q.off_bad = off;     off = align_up(off + sizeof(int64_t) * size_t(nblocks), kRegionAlign);
  q.off_offsets = off; off = align_up(off + sizeof(int64_t) * size_t(q.G + 1), kRegionAlign);
  q.off_rows = off;    off = align_up(off + sizeof(int32_t) * size_t(M), kRegionAlign);
  q.total = off;
  *p = q;
  return PGG_OK;
}

pgg_status make_unpermute_plan(const pgg_moe_unpermute_desc* d, UnpermutePlan* p) {
  if (!d || !p) return PGG_ERR_INVALID_ARG;
  if (d->reserved != 0 || d->batch <= 0 || d->topk <= 0 || d->hidden <= 0) return PGG_ERR_INVALID_ARG;
  if (d->row_idx_type != 0 && d->row_idx_type != 1) return PGG_ERR_INVALID_ARG;
  if (d->dtype < PGG_F32 || d->dtype > PGG_BF16) return PGG_ERR_INVALID_ARG;
  if (d->topk > INT64_MAX / d->batch) return PGG_ERR_INVALID_ARG;
  const int64_t M = d->batch * d->topk;
  if (M >= (int64_t(1) << 31) - 1 || d->batch >= (int64_t(1) << 31) ||
      d->hidden >= (int64_t(1) << 40) / M)
    return PGG_ERR_UNSUPPORTED;
  UnpermutePlan q{};
  q.M = M;
  q.batch = d->batch;
  q.topk = d->topk;
  q.H = d->hidden;
  q.dtype = d->dtype;
  q.row_idx_type = d->row_idx_type;
  size_t off = 0;
  q.off_header = off; off = align_up(off + sizeof(WsHeader), kRegionAlign);
  q.off_inv = off;    off = align_up(off + sizeof(int32_t) * size_t(M), kRegionAlign);
  q.off_ori = off;    off = align_up(off + sizeof(int32_t) * size_t(M), kRegionAlign);
  q.total = off;
  *p = q;
  return PGG_OK;
}

pgg_status make_dw_plan(const pgg_moe_fwd_desc* d, Plan* p) {
  Plan q;
  const pgg_status st = make_fwd_plan(d, &q);
  if (st != PGG_OK) return st;
  q.ksplit = 1;
  q.kspan = static_cast<int32_t>(q.N);
  q.ring_rows = 0;
  q.ring_bytes = 0;
  q.total = q.table_bytes;
  *p = q;
  return PGG_OK;
}

pgg_status check_gate_desc(const pgg_moe_gate_desc* d) {
  if (!d || d->reserved != 0) return PGG_ERR_INVALID_ARG;
  if (d->tokens <= 0 || d->experts <= 0 || d->topk <= 0 || d->topk > d->experts) return PGG_ERR_INVALID_ARG;
  if (d->renorm != 0 && d->renorm != 1) return PGG_ERR_INVALID_ARG;
  if (d->dtype < PGG_F32 || d->dtype > PGG_BF16) return PGG_ERR_INVALID_ARG;
  // the picks of a row live in registers, and a launch of up to 64 lanes per
  // row, in workgroups of 4 rows, holds fewer than 2^32 lanes
  if (d->experts > 8192 || d->topk > PGG_GATE_MAX_TOPK || d->tokens > (int64_t(1) << 26) - 4)
    return PGG_ERR_UNSUPPORTED;
  return PGG_OK;
}

namespace {

// Splits of a reduction of n elements for `busy` tiles: enough that about
// `target` workgroups run, each with at least min_span elements (a multiple of 64).
template <class Span>
void split_reduction(int64_t n, int64_t busy, int64_t target, int64_t min_span, int32_t* ksplit, Span* kspan) {
  constexpr int64_t kStage = 64, kMost = 64;
  int64_t split = std::min<int64_t>((target + busy / 2) / busy, n / min_span);
  split = std::max<int64_t>(1, std::min<int64_t>(split, kMost));
  const int64_t span = ((n + split - 1) / split + kStage - 1) / kStage * kStage;
  *kspan = static_cast<Span>(span);
  *ksplit = static_cast<int32_t>((n + span - 1) / span);
}

// Rows that are not 16-byte aligned can be copied to padded ones (whole 128-byte
// lines), which lets the large direct-to-LDS tiles take them instead of the
// tiles that load through registers.  An activation row is read by many columns
// and always pays for its copy.  Weights pay from this many rows per matrix on.
// Measured in us, bf16, without and with the copy:
//   gated product, 16 experts, K 4095, F 2047: 256 rows per expert 388, 462;
//     512 633, 577; 1024 1128, 803
//   its gradient, 16 experts, D 4095, F 2048: 128 rows per expert 180, 225;
//     256 285, 257; 1024 715, 506
//   adapters, 4095 x 4095: 1024 tokens 94, 108; 4096 294, 235
constexpr int64_t kPadRowsGlu = 512, kPadRowsGluGrad = 256, kPadRowsLora = 2048;
int64_t pad_pitch(int64_t len) { return (len + 63) / 64 * 64; }

}  // namespace

pgg_status make_glu_plan(const pgg_moe_glu_desc* d, Plan* p) {
  if (!d || !p) return PGG_ERR_INVALID_ARG;
  if (d->act != PGG_ACT_SILU && d->act != PGG_ACT_GELU_TANH) return PGG_ERR_INVALID_ARG;
  if (d->weight_cols % 2 != 0) return PGG_ERR_INVALID_ARG;
  pgg_moe_fwd_desc f = {};
  f.x_rows = d->x_rows;
  f.x_cols = d->x_cols;
  f.weight_groups = d->weight_groups;
  f.weight_rows = d->weight_rows;
  f.weight_cols = d->weight_cols;
  f.idx_len = d->idx_len;
  f.group_list_len = d->group_list_len;
  f.batch = d->batch;
  f.topk = d->topk;
  f.row_idx_type = d->row_idx_type;
  f.x_dtype = d->x_dtype;
  f.weight_dtype = d->weight_dtype;
  const pgg_status st = make_fwd_plan(&f, p);
  if (st != PGG_OK) return st;
  // the kernels count the reduction in 32 bits, up to three stages past its end
  if (d->x_cols > (int64_t(1) << 31) - 256) return PGG_ERR_UNSUPPORTED;
  // tiles of 128 rows and 128 columns where rows are not 16-byte aligned are four
  // times as many as the plan's; a launch holds fewer than 2^32 lanes
  if (int64_t(p->max_tiles) * p->n_col_tiles >= (int64_t(1) << 21)) return PGG_ERR_UNSUPPORTED;
  p->fused_prep = p->M <= 1024;
  // Few rows per expert: m-tiles of 32 or 64 rows x 256 columns (128 of h), two
  // workgroups per compute unit; otherwise one of the large tiles, or two of
  // 128 x 128.  Where tiles alone do not fill the chip, the reduction is split.
  // An expert of more rows than a tile reads its weights again, and the tiles of
  // 64 rows have to be direct-to-LDS ones.  Measured in us, 32 and 64 rows:
  //   bf16, 16 experts, K 4096, F 2048: 24 rows per expert 99, 99; 32 142, 101;
  //     48 156, 107; 60 186, 149
  //   K 4095, F 2047: 24 126, 150; 32 172, 151; 48 163, 155; 60 239, 247
  //   f32, K 2048, F 1408: 24 95, 173; 32 121, 175; 48 168, 175; 60 170, 178
  const int64_t cus = p->regime == kLarge ? 256 : 512;
  if (p->M <= 64 * p->G) {
    p->regime = kStream;
    const bool rows16 = p->dtype != PGG_F32 && p->N % 8 == 0 && p->K % 16 == 0;
    p->bm = !rows16 || p->M <= 24 * p->G ? 32 : 64;
    p->bn = 256;
    p->max_tiles = static_cast<int32_t>((p->M + p->bm - 1) / p->bm + p->G);
    p->n_col_tiles = static_cast<int32_t>((p->K + 255) / 256);
  }
  p->max_tiles = static_cast<int32_t>(std::min<int64_t>(p->max_tiles, p->M));   // each holds a row at least
  const int64_t busy = std::min<int64_t>(p->max_tiles, p->M / p->bm + (p->G + 1) / 2 + 1) * p->n_col_tiles;
  split_reduction(p->N, busy, p->regime == kStream ? 512 : cus,
                  p->regime != kStream ? 256 : p->dtype == PGG_F32 ? 32 : 128, &p->ksplit, &p->kspan);
  // few groups and rows: every workgroup finds its own tile (pgg_local.h)
  p->local = p->regime == kStream && p->G <= kLocalGroups && p->M <= kLocalRows;
  p->tc = p->max_tiles;
  size_t off = p->off_tiles;
  off = align_up(off + sizeof(MTile) * size_t(p->max_tiles), kRegionAlign);
  p->off_chunks = off;   off = align_up(off + sizeof(int32_t) * size_t(p->max_chunks + 1), kRegionAlign);
  p->off_inv = off;      off = align_up(off + sizeof(int32_t) * size_t(p->M), kRegionAlign);
  p->off_ori = off;      off = align_up(off + sizeof(int32_t) * size_t(p->M), kRegionAlign);
  p->table_bytes = p->off_ring = off;
  p->ring_bytes = p->ksplit > 1 ? size_t(p->ksplit) * size_t(p->M) * size_t(p->K) * sizeof(float) : 0;
  p->ring_rows = 0;
  off = align_up(off + p->ring_bytes, kRegionAlign);
  p->lda = p->N;
  p->ldw = p->K;
  p->off_pad_a = p->off_pad_w = off;
  if (p->regime == kLarge) {
    const int64_t F = p->K / 2, per_expert = p->M / p->G;
    const bool w_pays = F % 8 == 0 || per_expert >= kPadRowsGlu;
    p->pad_a = p->N % 8 != 0 && w_pays;
    p->pad_w = F % 8 != 0 && w_pays;
    if (p->pad_a) {
      p->lda = pad_pitch(p->N);
      off = align_up(off + size_t(p->batch) * size_t(p->lda) * 2, kRegionAlign);
    }
    p->off_pad_w = off;
    if (p->pad_w) {
      p->ldw = 2 * pad_pitch(F);
      off = align_up(off + size_t(p->G) * size_t(p->N) * size_t(p->ldw) * 2, kRegionAlign);
    }
  }
  p->total = off;
  return PGG_OK;
}

pgg_status make_glu_grad_plan(const pgg_moe_glu_grad_desc* d, Plan* p) {
  if (!d || !p || d->reserved != 0) return PGG_ERR_INVALID_ARG;
  if (d->act != PGG_ACT_SILU && d->act != PGG_ACT_GELU_TANH) return PGG_ERR_INVALID_ARG;
  if (d->grad_y_dtype != d->weight_dtype) return PGG_ERR_INVALID_ARG;
  if (d->grad_y_dtype < PGG_F32 || d->grad_y_dtype > PGG_BF16) return PGG_ERR_INVALID_ARG;
  const int64_t M = d->grad_y_rows, D = d->grad_y_cols, G = d->weight_groups, F = d->weight_rows;
  if (M <= 0 || D <= 0 || G <= 0 || F <= 0) return PGG_ERR_INVALID_ARG;
  if (D != d->weight_cols || d->group_list_len != G) return PGG_ERR_INVALID_ARG;
  if (M >= (int64_t(1) << 31) - 1 || G >= (int64_t(1) << 30) || D >= (int64_t(1) << 31) ||
      F >= (int64_t(1) << 30))
    return PGG_ERR_UNSUPPORTED;
  Plan q{};
  q.M = M; q.N = D; q.G = G; q.K = F; q.batch = M; q.topk = 1;
  q.panel_cols = F;
  q.dtype = d->grad_y_dtype;
  q.regime = q.dtype == PGG_F32 ? kF32 : kLarge;
  // m-tiles of 32 rows, 64 or the large ones.  Measured in us, whole calls, 32 and
  // 64 rows, F 1408 and 16 experts where not stated:
  //   bf16, D 4096: 24 rows per expert 53, 61; 32 57, 65; 36 69, 65; 48 72, 58; 60 77, 62
  //   D 4095: 24 73, 77; 32 75, 89; 36 101, 91; 48 103, 82; 60 109, 86
  //   D 7168, F 2048, 60 experts: 32 355, 388; 36 429, 396; 60 467, 428
  //   f32, D 2048: 32 63, 103; 40 96, 105; 48 98, 92; 60 98, 94
  q.bm = M <= (q.dtype == PGG_F32 ? 40 : 32) * G ? 32 : M <= 64 * G ? 64 : q.dtype == PGG_F32 ? 128 : 256;
  q.bn = 128;
  const int64_t max_tiles = std::min<int64_t>(M, (M + q.bm - 1) / q.bm + G);   // each holds a row at least
  const int64_t col_tiles = (F + q.bn - 1) / q.bn;
  // launches of fewer than 2^32 lanes, also as tiles of 128 rows
  if (max_tiles * col_tiles >= (int64_t(1) << 22)) return PGG_ERR_UNSUPPORTED;
  q.max_tiles = static_cast<int32_t>(max_tiles);
  q.tc = q.max_tiles;
  q.max_chunks = 1;
  q.n_panels = 1;
  q.n_col_tiles = static_cast<int32_t>(col_tiles);
  // Where tiles alone do not fill the chip (one 256 x 256 tile, two of 128 x
  // 128, three of 64 x 128 or four of 32 x 128 per compute unit), the reduction is split.
  q.local = q.bm <= 64 && G <= kLocalGroups;   // few groups: every workgroup finds its own tile (pgg_local.h)
  const int64_t busy_cols = q.bm == 256 ? (F + 255) / 256 : col_tiles;
  const int64_t busy = std::min<int64_t>(max_tiles, M / q.bm + (G + 1) / 2 + 1) * busy_cols;
  const int64_t fill = q.bm == 256 ? 256 : q.bm == 128 ? 512 : q.bm == 64 ? 768 : 1024;
  split_reduction(D, busy, fill, q.bm <= 64 ? 128 : 256, &q.ksplit, &q.kspan);
  size_t off = 0;
  q.off_header = off;   off = align_up(off + sizeof(WsHeader), kRegionAlign);
  q.off_offsets = off;  off = align_up(off + sizeof(int64_t) * size_t(G + 1), kRegionAlign);
  q.off_tiles = off;    off = align_up(off + sizeof(MTile) * size_t(q.max_tiles), kRegionAlign);
  q.off_chunks = off;   off = align_up(off + sizeof(int32_t) * 2, kRegionAlign);
  q.off_inv = q.off_ori = q.off_ring = off;
  q.table_bytes = off;
  if (q.ksplit > 1) off = align_up(off + size_t(q.ksplit) * size_t(M) * size_t(F) * sizeof(float), kRegionAlign);
  q.lda = q.ldw = D;
  q.off_pad_a = q.off_pad_w = off;
  q.pad_a = q.pad_w = q.bm == 256 && D % 8 != 0 && M / G >= kPadRowsGluGrad;
  if (q.pad_a) {
    q.lda = q.ldw = pad_pitch(D);
    off = align_up(off + size_t(M) * size_t(q.lda) * 2, kRegionAlign);
    q.off_pad_w = off;
    off = align_up(off + size_t(G) * size_t(F) * size_t(q.ldw) * 2, kRegionAlign);
  }
  q.total = off;
  *p = q;
  return PGG_OK;
}

pgg_status make_lora_plan(const pgg_lora_desc* d, LoraPlan* p) {
  if (!d || !p || d->reserved != 0) return PGG_ERR_INVALID_ARG;
  if (d->tokens <= 0 || d->in_features <= 0 || d->out_features <= 0 || d->adapters <= 0 || d->rank <= 0)
    return PGG_ERR_INVALID_ARG;
  if (d->dtype < PGG_F32 || d->dtype > PGG_BF16) return PGG_ERR_INVALID_ARG;
  if (d->tokens >= (int64_t(1) << 31) - 1 || d->in_features >= (int64_t(1) << 31) ||
      d->out_features >= (int64_t(1) << 31) || d->adapters >= (int64_t(1) << 31) || d->rank > PGG_LORA_MAX_RANK)
    return PGG_ERR_UNSUPPORTED;
  LoraPlan q{};
  q.T = d->tokens;
  q.K = d->in_features;
  q.N = d->out_features;
  q.P = d->adapters;
  q.rank = static_cast<int32_t>(d->rank);
  q.dtype = d->dtype;
  const bool f32 = q.dtype == PGG_F32;
  auto tiles = [&](int64_t bm, int64_t bn) { return ((q.T + bm - 1) / bm) * ((q.N + bn - 1) / bn); };
  // launches of fewer than 2^32 lanes: 256 per tile at least, and 4096 per 256
  // tokens for z, with one workgroup of 512 more
  if (tiles(32, 128) >= (int64_t(1) << 23) || q.T > (int64_t(1) << 28) - 256) return PGG_ERR_UNSUPPORTED;
  // With few tokens the projection is bound by reading W: tiles of 32 or 64 rows,
  // the reduction split over about 512 workgroups, two per compute unit.  Above
  // that, the 256 x 256 tiles (one workgroup per compute unit) or the 128 x 128
  // ones (two), split where there are too few of them.  Measured in us, 96, 128,
  // 192 and 256 tokens, the large tiles and the small ones:
  //   bf16, 4096 x 4096: 34, 31; 36, 34; 42, 43; 47, 46
  //   4096 x 192:        24, 15; 24, 16; 27, 17; 29, 21
  //   4095 x 4095:       38, 34; 42, 42; 45, 47; 50, 57
  //   3977 x 190:        22, 17; 23, 19; 25, 23; 25, 28
  //   f32, 2048 x 1408:  38, 24; 38, 29; 40, 36; 41, 39
  q.few = q.T <= (f32 || (q.K % 8 == 0 && q.N % 8 == 0) ? 256 : 128);
  q.lda = q.K;
  q.ldw = q.N;
  const bool w_pays = q.N % 8 == 0 || q.T >= kPadRowsLora;
  q.pipe = !q.few && !f32 && w_pays;
  q.pad_a = q.pipe && q.K % 8 != 0;
  q.pad_w = q.pipe && q.N % 8 != 0;
  if (q.few) split_reduction(q.K, tiles(64, f32 ? 128 : 256), 512, 128, &q.ksplit, &q.kspan);
  else if (q.pipe) split_reduction(q.K, tiles(256, 256), 256, 256, &q.ksplit, &q.kspan);
  else split_reduction(q.K, tiles(128, 128), 512, 256, &q.ksplit, &q.kspan);
  size_t off = 0;
  q.off_header = off; off = align_up(off + sizeof(WsHeader), kRegionAlign);
  q.off_z = off;      off = align_up(off + sizeof(float) * size_t(q.T) * size_t(q.rank), kRegionAlign);
  q.off_part = off;
  if (q.few || q.ksplit > 1)
    off = align_up(off + sizeof(float) * size_t(q.ksplit) * size_t(q.T) * size_t(q.N), kRegionAlign);
  q.off_pad_a = off;
  if (q.pad_a) {
    q.lda = pad_pitch(q.K);
    off = align_up(off + size_t(q.T) * size_t(q.lda) * 2, kRegionAlign);
  }
  q.off_pad_w = off;
  if (q.pad_w) {
    q.ldw = pad_pitch(q.N);
    off = align_up(off + size_t(q.K) * size_t(q.ldw) * 2, kRegionAlign);
  }
  q.total = off;
  *p = q;
  return PGG_OK;
}

pgg_status check_gate_grouped_desc(const pgg_moe_gate_grouped_desc* d) {
  if (!d) return PGG_ERR_INVALID_ARG;
  if (d->tokens <= 0 || d->experts <= 0 || d->topk <= 0 || d->groups <= 0 || d->topk_groups <= 0)
    return PGG_ERR_INVALID_ARG;
  if (d->groups > d->experts || d->experts % d->groups != 0 || d->topk_groups > d->groups) return PGG_ERR_INVALID_ARG;
  const int64_t each = d->experts / d->groups;
  if ((d->topk + each - 1) / each > d->topk_groups) return PGG_ERR_INVALID_ARG;
  if (d->score != PGG_SCORE_SIGMOID && d->score != PGG_SCORE_SOFTMAX) return PGG_ERR_INVALID_ARG;
  if (d->renorm != 0 && d->renorm != 1) return PGG_ERR_INVALID_ARG;
  if (d->dtype < PGG_F32 || d->dtype > PGG_BF16) return PGG_ERR_INVALID_ARG;
  // as for the gate; the groups' scores live in LDS, one bit of a word each in the long form
  if (d->experts > 8192 || d->topk > PGG_GATE_MAX_TOPK || d->groups > PGG_GATE_MAX_GROUPS ||
      d->tokens > (int64_t(1) << 26) - 4)
    return PGG_ERR_UNSUPPORTED;
  return PGG_OK;
}

pgg_status make_w4_layout(const pgg_w4_desc* d, W4Layout* l) {
  if (!d || !l || d->reserved != 0) return PGG_ERR_INVALID_ARG;
  if (d->groups <= 0 || d->rows <= 0 || d->cols <= 0 || d->group_size <= 0) return PGG_ERR_INVALID_ARG;
  if (d->group_size != 32 && d->group_size != 64 && d->group_size % 128 != 0) return PGG_ERR_INVALID_ARG;
  if ((d->zeros != 0 && d->zeros != 1) || (d->gated != 0 && d->gated != 1)) return PGG_ERR_INVALID_ARG;
  if (d->gated && d->cols % 2 != 0) return PGG_ERR_INVALID_ARG;
  if (d->dtype < PGG_F32 || d->dtype > PGG_BF16) return PGG_ERR_INVALID_ARG;
  if (d->groups >= (int64_t(1) << 30) || d->rows > (int64_t(1) << 31) - 1024 || d->cols > (int64_t(1) << 31) - 1024)
    return PGG_ERR_UNSUPPORTED;
  W4Layout q{};
  q.G = d->groups;
  q.K = d->rows;
  q.N = d->cols;
  q.group_size = d->group_size;
  q.KB = static_cast<int32_t>((q.K + 127) / 128);
  q.CB = static_cast<int32_t>(d->gated ? (q.N / 2 + 31) / 32 : (q.N + 63) / 64);
  q.sub = d->group_size == 32 ? 4 : d->group_size == 64 ? 2 : 1;
  q.dtype = d->dtype;
  q.zeros = d->zeros;
  q.gated = d->gated;
  const int64_t plane = int64_t(q.KB) * q.CB;
  // 31-bit byte offsets within a matrix (codes, and fp32 scales of groups of 32)
  if (plane >= (int64_t(1) << 19) || plane * q.G >= (int64_t(1) << 40)) return PGG_ERR_UNSUPPORTED;
  q.tiles = plane * q.G;
  q.off_scales = size_t(q.tiles) * 4096;
  q.off_zeros = align_up(q.off_scales + size_t(q.tiles) * q.sub * 64 * (q.dtype == PGG_F32 ? 4 : 2), 256);
  q.total = align_up(q.off_zeros + (q.zeros ? size_t(q.tiles) * q.sub * 64 : 0), 256);
  *l = q;
  return PGG_OK;
}

pgg_status make_w4_plan(const pgg_moe_w4_desc* d, bool gated, W4Plan* p) {
  if (!d || !p) return PGG_ERR_INVALID_ARG;
  W4Plan w{};
  const pgg_status st = make_w4_layout(&d->weight, &w.layout);
  if (st != PGG_OK) return st;
  const W4Layout& l = w.layout;
  if (gated != (l.gated != 0)) return PGG_ERR_INVALID_ARG;
  if (d->act != PGG_ACT_SILU && d->act != PGG_ACT_GELU_TANH) return PGG_ERR_INVALID_ARG;
  if (d->topk <= 0 || d->batch <= 0 || d->x_rows != d->batch || d->x_cols != l.K) return PGG_ERR_INVALID_ARG;
  if (d->row_idx_type != 0 && d->row_idx_type != 1) return PGG_ERR_INVALID_ARG;
  if (d->group_list_len != l.G || d->topk > INT64_MAX / d->batch) return PGG_ERR_INVALID_ARG;
  const int64_t M = d->batch * d->topk;
  const bool indexed = d->idx_len != 0;
  if (indexed ? d->idx_len != M : d->topk != 1) return PGG_ERR_INVALID_ARG;
  if (M >= (int64_t(1) << 31) - 1) return PGG_ERR_UNSUPPORTED;
  Plan& q = w.base;
  q.M = M; q.N = l.K; q.G = l.G; q.K = l.N; q.batch = d->batch; q.topk = d->topk;
  q.row_idx_type = d->row_idx_type;
  q.dtype = l.dtype;
  q.n_panels = 1;
  q.max_chunks = 1;
  q.regime = kStream;
  // Rows of a tile.  An expert with more rows than a tile reads its weights again,
  // and one of 16-bit x with many multiplies faster in the 64 x 256 tiles; a token
  // goes to an expert once, so with an index no expert has more rows than there are
  // tokens.  Measured in us, 16 experts, tiles of 16, 32 and 64 rows:
  //   bf16, 7168 x 4096: 8 rows per expert 53, 60, 70; 16 62, 66, 69; 24 106, 73, 70;
  //     32 110, 82, 84; 48 161, 142, 85; 64 202, 150, 87; 1024 3258, 2268, 945
  //   f16, 1403 x 2039, groups of 64: 8 15, 23, 33; 32 28, 23, 35; 64 48, 39, 40; 128 86, 66, 41
  // How the rows are spread the host does not know, so the rule goes by their average
  // over all experts.  From 24 the 64 x 256 tiles lose little where experts are alike
  // and win where few have the rows, if the call is large: tiles of 32 rows would be
  // two workgroups to a compute unit (with an index, whose tables the large tiles
  // need, three).  Tiles of 32 and of 64 rows at 24 on average: experts drawn alike,
  // by a popularity of 1 / rank^1.1, and all rows on 2 experts:
  //   16, bf16, 7168 x 4096: 73 67, 92 101, 73 68;  64, 2048 x 2816: 75 59, 79 69, 67 42
  //   64, f16, 1403 x 2039: 64 41, 63 57, 43 38
  //   and of small matrices, 8, bf16, 1408 x 2048: 14 24, 14 25;  16, 512 x 512: 11 17, 11 18
  // (They address x with 32-bit byte offsets, padded rows included.)
  const bool large = (M + 31) / 32 * l.CB >= (indexed ? 768 : 512);
  w.tiles = l.dtype != PGG_F32 && (M > 32 * l.G || (large && M >= 24 * l.G)) && !(indexed && d->batch <= 32) &&
            d->batch < ((int64_t(1) << 31) - 64) / 2 / (l.K + 64);
  q.bm = w.tiles ? 64 : l.dtype == PGG_F32 || M <= 12 * l.G || (indexed && d->batch <= 16) ? 16 : 32;
  const int64_t max_tiles = std::min<int64_t>(M, (M + q.bm - 1) / q.bm + l.G);   // each holds a row at least
  const int64_t col_tiles = w.tiles ? (l.CB + 3) / 4 : l.CB;
  // Launches of fewer than 2^32 lanes: many tiles take 256 lanes to four column blocks
  // or what is left of them.
  if (max_tiles * ((l.CB + 3) / 4) >= (int64_t(1) << 24)) return PGG_ERR_UNSUPPORTED;
  q.max_tiles = static_cast<int32_t>(max_tiles);
  q.tc = q.max_tiles;
  // few groups: every workgroup finds its own tile (and, with a routing index, few rows)
  q.local = !w.tiles && l.G <= kLocalGroups && (!indexed || M <= kLocalRows);
  q.fused_prep = M <= 1024;
  const int64_t busy = std::min<int64_t>(max_tiles, M / q.bm + (l.G + 1) / 2 + 1) * col_tiles;
  w.sub = l.sub;
  // Tiles of few rows: about three waves to a SIMD.  With many column blocks one
  // wave takes the whole reduction, and four blocks side by side share their rows
  // of x in L1; with few the reduction is split over waves, and with very few over
  // workgroups.  Measured in us, waves per block x blocks side by side:
  //   4096 blocks, 7168 deep, 16 rows: 4x1 212, 2x2 201, 1x4 197; 2048: 109, 102, 99
  //   1024 blocks: 8 rows 48.6, 45.6, -; 16 rows 58.2, 53.2, -; 768: 37.3, 42.8, 53.0
  //   2048 blocks, 1408 deep, 12 rows: 37.6, 29.4, 26.7;  176, 2048 deep: 11.6, 16.9, 27.0, 8x1 11.1
  //   over workgroups (8x1, 4x1 with 4 splits): 32 blocks, 7168 deep 13.5, 11.2; 112 14.4, 13.6;
  //     22 blocks, 2048 deep 9.2, 11.7
  w.waves = busy >= 2048 ? 1 : busy >= 1280 ? 2 : busy >= 256 ? 4 : 8;
  w.beside = busy >= 2048 ? 4 : busy >= 1280 ? 2 : 1;
  int64_t split = 1;
  if (w.tiles) {   // two workgroups to a compute unit
    if (busy <= 256) split = std::min<int64_t>(std::min<int64_t>(512 / busy, l.KB / 8), 16);
  } else if (busy <= 128 && l.KB >= 28) {
    split = std::min<int64_t>(l.KB / 14, 4);
    w.waves = 4;
  }
  split = std::max<int64_t>(split, 1);
  w.kb_span = static_cast<int32_t>((l.KB + split - 1) / split);
  w.ksplit = (l.KB + w.kb_span - 1) / w.kb_span;
  q.ksplit = w.ksplit;
  size_t off = 0;
  q.off_header = off;   off = align_up(off + sizeof(WsHeader), kRegionAlign);
  q.off_offsets = off;  off = align_up(off + sizeof(int64_t) * size_t(l.G + 1), kRegionAlign);
  q.off_tiles = off;    off = align_up(off + sizeof(MTile) * size_t(q.max_tiles), kRegionAlign);
  q.off_chunks = off;   off = align_up(off + sizeof(int32_t) * 2, kRegionAlign);
  q.off_inv = off;      off = align_up(off + (indexed ? sizeof(int32_t) * size_t(M) : 0), kRegionAlign);
  q.off_ori = off;      off = align_up(off + (indexed ? sizeof(int32_t) * size_t(M) : 0), kRegionAlign);
  q.table_bytes = q.off_ring = off;
  if (w.ksplit > 1) off = align_up(off + size_t(w.ksplit) * size_t(M) * 64 * size_t(l.CB) * sizeof(float), kRegionAlign);
  // x is read in chunks of 16 bytes: rows that end inside one are copied to longer
  // ones.  (Read where they lie, at odd addresses, rows of 1403 f16 elements made a
  // call of 36 us with its copy take 57.)
  const int64_t chunk = l.dtype == PGG_F32 ? 4 : 8;
  q.lda = l.K;
  q.off_pad_a = off;
  q.pad_a = l.K % chunk != 0;
  if (q.pad_a) {
    q.lda = pad_pitch(l.K);
    off = align_up(off + size_t(q.batch) * size_t(q.lda) * (l.dtype == PGG_F32 ? 4 : 2), kRegionAlign);
  }
  w.off_sums = off;
  if (w.tiles) off = align_up(off + sizeof(float) * size_t(q.batch) * size_t(l.KB) * l.sub, kRegionAlign);
  q.total = off;
  *p = w;
  return PGG_OK;
}

pgg_status make_combine_plan(const pgg_moe_combine_desc* d, CombinePlan* p) {
  if (!d || !p) return PGG_ERR_INVALID_ARG;
  if (d->batch <= 0 || d->topk <= 0 || d->hidden <= 0) return PGG_ERR_INVALID_ARG;
  if (d->row_idx_type != 0 && d->row_idx_type != 1) return PGG_ERR_INVALID_ARG;
  if (d->dtype < PGG_F32 || d->dtype > PGG_BF16) return PGG_ERR_INVALID_ARG;
  if (!(d->eps >= 0.0f) || d->topk > INT64_MAX / d->batch) return PGG_ERR_INVALID_ARG;
  const int64_t M = d->batch * d->topk;
  // a workgroup of 512 threads takes four pieces of 8 elements to a thread; a
  // launch holds fewer than 2^32 lanes
  if (M >= (int64_t(1) << 31) - 1 || d->hidden > 16384) return PGG_ERR_UNSUPPORTED;
  CombinePlan q{};
  q.M = M;
  q.batch = d->batch;
  q.topk = d->topk;
  q.H = d->hidden;
  q.alpha = d->residual_scale;
  q.eps = d->eps;
  q.dtype = d->dtype;
  q.row_idx_type = d->row_idx_type;
  q.row_long = q.H > 8192;
  if ((q.batch + 1024) * q.threads(false) >= (int64_t(1) << 32)) return PGG_ERR_UNSUPPORTED;
  // the gradient's workgroups, one or more to a compute unit, go through the tokens
  q.grad_blocks = std::min<int64_t>(q.batch, 256 * (512 / q.threads(true)));
  size_t off = 0;
  q.off_header = off; off = align_up(off + sizeof(WsHeader), kRegionAlign);
  q.off_inv = off;    off = align_up(off + sizeof(int32_t) * size_t(M), kRegionAlign);
  q.off_ori = off;    off = align_up(off + sizeof(int32_t) * size_t(M), kRegionAlign);
  q.off_part = q.total_fwd = off;
  q.total_grad = align_up(off + 2 * size_t(q.grad_blocks) * size_t(q.H) * sizeof(float), kRegionAlign);
  *p = q;
  return PGG_OK;
}

}  // namespace pgg
