// muon.hip -- the entry points of the orthogonalisation and of the step that
// takes it (fp_muon_*): argument checks, plans, their device tables, the
// iteration's scales.  Every check runs before anything is enqueued.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>
#include <vector>

#include "fp_matrix.h"
#include "plan_util.h"

using namespace fpk;

namespace {

constexpr int64_t kMaxSide = 1 << 20;

int64_t dtype_bytes(int32_t dtype) { return dtype == FP_DTYPE_F32 ? 4 : 2; }

// The matrices of a batch share every launch and the workspace.  A batch is
// closed once it holds this much of it.
constexpr int64_t kBatchBytes = (int64_t)1 << 31;

// Tiles [first, first + n) of the plan's table.
struct Run {
    int64_t first = 0, n = 0;
};

// Of matrices, how many small ones are few beside large ones (create()), and how many
// are few for a launch of their own (group_small()).
constexpr int64_t kFewSmall = 128, kFewForLaunch = 512;

// Small matrices that need about as much: one launch.
struct Small {
    Run run;
    int tiles = 0;
    unsigned lds = 0;
};

struct Batch {
    std::vector<int32_t> mats;
    Run moment, norm, cast, gram, join, half, full;
    int gram_shape = kTile64, half_shape = kTile64, full_shape = kTile64;
};

}  // namespace

struct fp_muon {
    int32_t n = 0;
    int device = -1;
    int32_t grad_dtype = FP_DTYPE_F32, copy_dtype = FP_DTYPE_BF16, update_dtype = FP_DTYPE_BF16;
    bool has_master = false, has_update = false;
    int32_t max_group = 0;
    int64_t partition = 0, workspace = 0;
    std::vector<int64_t> numel, offset;
    std::vector<Batch> batches;
    std::vector<Small> smalls;
    std::vector<Span> written;         // weights, copies and updates
    void* dev = nullptr;               // records, gradient table, tile table
    void* staging = nullptr;           // pinned, of the gradient table's uploads
    hipEvent_t uploaded = nullptr;
    std::mutex mu;                     // guards the gradients: their table's upload and
    std::vector<Span> read;            // where they lie

    const MuonRec* recs() const { return static_cast<const MuonRec*>(dev); }
    const void** grads() const { return reinterpret_cast<const void**>(static_cast<char*>(dev) + sizeof(MuonRec) * (size_t)n); }
    const MatTile* tile_table() const { return reinterpret_cast<const MatTile*>(grads() + (n + 1) / 2 * 2); }
};

namespace {

void free_plan(fp_muon* p) {
    int cur = -1;
    (void)hipGetDevice(&cur);
    if (p->device >= 0) (void)hipSetDevice(p->device);
    if (p->uploaded) (void)hipEventSynchronize(p->uploaded), (void)hipEventDestroy(p->uploaded);
    if (p->staging) (void)hipHostFree(p->staging);
    if (p->dev) (void)hipFree(p->dev);
    if (cur >= 0) (void)hipSetDevice(cur);
    delete p;
}

fp_status check_device(const fp_muon* p) {
    int device = -1;
    hipError_t e = hipGetDevice(&device);
    if (e != hipSuccess) return device_error(e, "hipGetDevice");
    if (device != p->device)
        return bad(FP_ERR_INVALID, "muon plan was created on device %d, current is %d", p->device, device);
    return FP_OK;
}

fp_status check_grads(const std::vector<int64_t>& numel, int32_t dtype, const std::vector<Span>& written,
                      const void* const* grads, std::vector<Span>* spans) {
    const int64_t es = dtype_bytes(dtype);
    std::vector<Span> v;
    for (size_t i = 0; i < numel.size(); ++i) {
        if (numel[i] == 0) continue;
        if (grads[i] == nullptr) return bad(FP_ERR_INVALID, "grads[%zu] is NULL", i);
        if (!on(grads[i], (uintptr_t)es)) return bad(FP_ERR_ALIGN, "grads[%zu] misaligned", i);
        v.push_back(span_of(grads[i], numel[i] * es));
        if (meets_any(v.back(), written)) return bad(FP_ERR_INVALID, "grads[%zu] overlaps a weight, a copy or an update", i);
    }
    *spans = joined(std::move(v));
    return FP_OK;
}

// Lays the matrix out in the workspace from byte `at` on; returns its end.
int64_t lay_out(MuonRec* r, int64_t at) {
    auto take = [&](int64_t bytes) {
        const int64_t from = at;
        at += ceil_div64(bytes, 256) * 256;
        return from;
    };
    const int64_t all = (int64_t)r->rp * r->cp, m = std::min(r->rp, r->cp);
    r->h[0] = take(2 * all);
    r->h[1] = take(2 * all);
    r->l = take(2 * all);
    r->a = take(2 * m * m);
    r->b = take(2 * m * m);
    r->da = take(4 * m);
    r->db = take(4 * m);
    r->part = take(8 * (r->chunks + 1));
    return at;
}

// Neighbouring tiles of one matrix's product, and the steps along K of each.
struct Chunk {
    int32_t mat;
    int64_t steps;
    std::vector<MatTile> tiles;
};

// The tiles of one matrix in an order in which neighbours read the same rows
// and columns: bands of four rows, column by column.  half: those on and below
// the diagonal of the smaller side's square.
std::vector<MatTile> ordered(const MuonRec& r, int32_t mat, int side, bool half) {
    const int64_t m = std::min(r.rp, r.cp);
    const int32_t rows = (int32_t)ceil_div64(half ? m : r.rp, side), cols = (int32_t)ceil_div64(half ? m : r.cp, side);
    std::vector<MatTile> v;
    for (int32_t band = 0; band < rows; band += 4)
        for (int32_t j = 0; j < cols; ++j)
            for (int32_t i = band; i < std::min(rows, band + 4); ++i)
                if (!half || j <= i) v.push_back({mat, i, j, 0});
    return v;
}

// A batch's product on tiles of one shape: when would its last workgroup end?
// In us, from what one step of a tile takes when its CU is full and when it is
// alone there, and from what a tile takes beside its steps (MI355X, the tiles'
// kernels at 1024 to 4096).
double finish(const std::vector<MuonRec>& recs, const Batch& b, int shape, bool half) {
    constexpr double kStep[] = {1.6, 0.56, 0.26, 0.4, 1.2}, kAlone[] = {1.3, 0.65, 0.36, 0.2, 1.2},
                     kBeside[] = {20.0, 6.0, 2.5, 3.0, 14.0};
    std::vector<std::pair<int64_t, int64_t>> runs;  // steps, tiles
    for (int32_t i : b.mats) {
        const MuonRec& r = recs[(size_t)i];
        const int64_t m = std::min(r.rp, r.cp), n = std::max(r.rp, r.cp), t = ceil_div64(m, kTileSide[shape]);
        runs.push_back({(half ? n : m) / 64, half ? t * (t + 1) / 2 : t * ceil_div64(n, kTileSide[shape])});
    }
    std::sort(runs.rbegin(), runs.rend());
    size_t kept = 0;  // runs of as many steps are one
    for (size_t i = 1; i < runs.size(); ++i) {
        if (runs[i].first == runs[kept].first) runs[kept].second += runs[i].second;
        else runs[++kept] = runs[i];
    }
    runs.resize(kept + 1);
    constexpr int kCus = 256;
    double load[kCus] = {};
    int64_t held[kCus] = {};
    double alone = 0.0;
    for (const auto& run : runs) {
        const double c = kStep[shape] * (double)run.first + kBeside[shape];
        alone = std::max(alone, kAlone[shape] * (double)run.first + kBeside[shape]);
        int64_t left = run.second;
        const int64_t each = left / kCus > 4 ? left / kCus - 2 : 0;  // most of a long run goes everywhere alike
        for (int k = 0; k < kCus; ++k) load[k] += c * (double)each, held[k] += each;
        for (left -= each * kCus; left > 0; --left) {
            const int k = (int)(std::min_element(load, load + kCus) - load);
            load[k] += c;
            ++held[k];
        }
    }
    double end = alone;
    for (int k = 0; k < kCus; ++k)
        if (held[k] > 1) end = std::max(end, load[k]);
    return end;
}

int choose_shape(const std::vector<MuonRec>& recs, const Batch& b, bool half) {
    int best = kTile256;
    for (int shape = kTile128; shape < (half ? kHalfShapes : kFullShapes); ++shape)
        if (finish(recs, b, shape, half) < finish(recs, b, best, half)) best = shape;
    return best;
}

// The table of a product.  The hardware deals workgroups out to the 8 dies in
// turn, each with an L2 of its own: entry 8 i + d is die d's i-th tile.  Runs of
// neighbours go to the die with the least work so far, the longest tiles first.
// sliced: A's, of which a matrix's slices are apart.
void deal(const std::vector<MuonRec>& recs, const Batch& b, int side, bool half, bool sliced, std::vector<MatTile>* table) {
    constexpr int kDies = 8;
    std::vector<Chunk> chunks;
    int64_t total = 0;
    for (int32_t i : b.mats) {
        const MuonRec& r = recs[(size_t)i];
        const bool slices = sliced && r.slices > 1;
        for (int32_t k = 0; k < (slices ? r.slices : 1); ++k) {
            Chunk c = {i, slices ? r.slice_steps : (half ? std::max(r.rp, r.cp) : std::min(r.rp, r.cp)) / 64, ordered(r, i, side, half)};
            for (MatTile& t : c.tiles) t.slice = k;
            total += (int64_t)c.tiles.size();
            chunks.push_back(std::move(c));
        }
    }
    std::stable_sort(chunks.begin(), chunks.end(), [](const Chunk& x, const Chunk& y) { return x.steps > y.steps; });
    std::vector<MatTile> die[kDies];
    int64_t load[kDies] = {};
    for (const Chunk& c : chunks)
        for (int64_t at = 0, n; at < (int64_t)c.tiles.size(); at += n) {
            // ever shorter towards the end, so that the shares come out alike
            n = std::min({(int64_t)c.tiles.size() - at, (int64_t)32, std::max<int64_t>(1, total / (4 * kDies))});
            total -= n;
            const int d = (int)(std::min_element(load, load + kDies) - load);
            load[d] += c.steps * n;
            die[d].insert(die[d].end(), c.tiles.begin() + at, c.tiles.begin() + (at + n));
        }
    size_t rows = 0;
    for (const auto& d : die) rows = std::max(rows, d.size());
    for (size_t i = 0; i < rows; ++i)
        for (const auto& d : die) table->push_back(i < d.size() ? d[i] : MatTile{-1, 0, 0, 0});
}

int64_t half_tiles(const MuonRec& r, int side) {
    const int64_t t = ceil_div64(std::min(r.rp, r.cp), side);
    return t * (t + 1) / 2;
}

// Where few tiles of A contract long rows, most CUs would be idle: the rows are cut
// into slices, and one launch more adds their sums up (five steps of 40 x 70000: 182
// us, else 1166; of 64 x 8192 110 and 218; of 28 matrices of 16 x 4096 174 and 219).
// Slices are as short as gives every one a CU to itself, and worth it where that
// ends earlier by more than the launch takes.  Returns whether there are any, and
// lays their sums out from byte *at on.
bool slice_gram(std::vector<MuonRec>* recs, const Batch& b, int64_t* at) {
    constexpr double kJoin = 6.0, kStep = 0.2, kBeside = 3.0;  // us; of the deep tiles
    constexpr int64_t kCus = 256;
    const int side = kTileSide[kTile64Deep];
    int64_t longest = 0, tiles = 0;
    for (int32_t i : b.mats) {
        const MuonRec& r = (*recs)[(size_t)i];
        longest = std::max<int64_t>(longest, std::max(r.rp, r.cp) / 64);
        tiles += half_tiles(r, side);
    }
    if (tiles > kCus) return false;
    int64_t steps = std::max<int64_t>(4, ceil_div64(longest, kMaxSlices));
    for (;; ++steps) {
        int64_t slots = 0;
        for (int32_t i : b.mats) {
            const MuonRec& r = (*recs)[(size_t)i];
            slots += half_tiles(r, side) * ceil_div64(std::max(r.rp, r.cp) / 64, steps);
        }
        if (slots <= kCus) break;  // ends: one slice each are no more than the tiles
    }
    if (kStep * (double)steps + kBeside + kJoin >= finish(*recs, b, b.half_shape, true)) return false;
    for (int32_t i : b.mats) {
        MuonRec& r = (*recs)[(size_t)i];
        r.slices = (int32_t)ceil_div64(std::max(r.rp, r.cp) / 64, steps);
        r.slice_steps = (int32_t)steps;
        r.split = *at;
        if (r.slices > 1) *at += (int64_t)r.slices * half_tiles(r, side) * side * side * 4;
    }
    return true;
}

// Closes a batch: its tiles, appended to the table; *at: the end of its workspace.
void close_batch(std::vector<MuonRec>* all, Batch* b, int64_t* at, std::vector<MatTile>* table) {
    const std::vector<MuonRec>& recs = *all;
    auto run = [&](Run* r, auto&& fill) {
        r->first = (int64_t)table->size();
        fill();
        r->n = (int64_t)table->size() - r->first;
    };
    auto grid = [&](auto&& rows, auto&& cols) {
        for (int32_t i : b->mats)
            for (int64_t ti = 0; ti < rows(recs[(size_t)i]); ++ti)
                for (int64_t tj = 0; tj < cols(recs[(size_t)i]); ++tj) table->push_back({i, (int32_t)ti, (int32_t)tj, 0});
    };
    run(&b->moment, [&] { grid([](const MuonRec& r) { return (int64_t)r.chunks; }, [](const MuonRec&) { return (int64_t)1; }); });
    run(&b->norm, [&] { grid([](const MuonRec& r) { return (int64_t)(r.chunks > kOwnChunks); }, [](const MuonRec&) { return (int64_t)1; }); });
    run(&b->cast, [&] {
        grid([](const MuonRec& r) { return ceil_div64(r.rp, kCastRows); }, [](const MuonRec& r) { return ceil_div64(r.cp, kCastCols); });
    });
    b->half_shape = choose_shape(recs, *b, true);
    b->full_shape = choose_shape(recs, *b, false);
    run(&b->half, [&] { deal(recs, *b, kTileSide[b->half_shape], true, false, table); });
    run(&b->full, [&] { deal(recs, *b, kTileSide[b->full_shape], false, false, table); });
    b->gram = b->half;
    b->gram_shape = b->half_shape;
    if (!slice_gram(all, *b, at)) return;
    b->gram_shape = kTile64Deep;
    run(&b->gram, [&] { deal(recs, *b, kTileSide[kTile64Deep], true, true, table); });
    run(&b->join, [&] {
        for (int32_t i : b->mats)
            if (recs[(size_t)i].slices > 1)
                for (const MatTile& t : ordered(recs[(size_t)i], i, kTileSide[kTile64Deep], true)) table->push_back(t);
    });
}

// The small matrices by what they need, largest first, in launches: a new one
// where a matrix needs half as much as the launch's first or less (its LDS
// decides how many workgroups a CU holds, its tiles how many registers), but not
// for the few that a launch of their own would cost more than it saves (one of 160 x
// 160 and 512 of 32 x 48: 81 us in one launch, 93 in two; 1024 of them 118 and 98, 4096
// 385 and 141; with 64 x 64 82 and 102, 131 and 116, 428 and 204).
std::vector<Small> group_small(const std::vector<MuonRec>& recs, std::vector<int32_t> mats, std::vector<MatTile>* table) {
    auto lds = [&](int32_t i) { return small_lds(recs[(size_t)i].rows, recs[(size_t)i].cols); };
    auto tiles = [&](int32_t i) { return small_tiles(recs[(size_t)i].rows, recs[(size_t)i].cols); };
    std::stable_sort(mats.begin(), mats.end(), [&](int32_t x, int32_t y) { return lds(x) > lds(y); });
    std::vector<Small> v;
    for (size_t at = 0; at < mats.size(); ++at) {
        const int32_t i = mats[at];
        if (v.empty() || (2 * lds(i) <= (int64_t)v.back().lds && (int64_t)(mats.size() - at) > kFewForLaunch)) {
            Small s;
            s.run.first = (int64_t)table->size();
            s.lds = (unsigned)lds(i);
            v.push_back(s);
        }
        Small& s = v.back();
        s.tiles = std::max(s.tiles, (int)tiles(i));
        ++s.run.n;
        table->push_back({i, 0, 0, 0});
    }
    return v;
}

fp_status create(int32_t n, const int64_t* rows, const int64_t* cols, const int32_t* group, int32_t grad_dtype,
                 const void* const* grads, float* const* master, int32_t copy_dtype, void* const* copies,
                 int32_t update_dtype, void* const* updates, fp_muon** out) {
    if (out == nullptr) return bad(FP_ERR_INVALID, "out is NULL");
    *out = nullptr;
    if (n < 1) return bad(FP_ERR_RANGE, "n must be >= 1");
    if (rows == nullptr || cols == nullptr || grads == nullptr) return bad(FP_ERR_INVALID, "rows, cols or grads is NULL");
    if (grad_dtype < FP_DTYPE_F32 || grad_dtype > FP_DTYPE_F16) return bad(FP_ERR_INVALID, "unknown grad_dtype %d", grad_dtype);
    if (copies != nullptr && copy_dtype != FP_DTYPE_BF16 && copy_dtype != FP_DTYPE_F16)
        return bad(FP_ERR_INVALID, "copy_dtype must be bf16 or fp16 (got %d)", copy_dtype);
    if (updates != nullptr && (update_dtype < FP_DTYPE_F32 || update_dtype > FP_DTYPE_F16))
        return bad(FP_ERR_INVALID, "unknown update_dtype %d", update_dtype);
    if (copies != nullptr && master == nullptr) return bad(FP_ERR_INVALID, "copies need master weights");
    if (master == nullptr && updates == nullptr) return bad(FP_ERR_INVALID, "neither master weights nor updates");
    std::vector<MuonRec> recs((size_t)n);
    std::vector<MatTile> table;
    std::vector<Batch> batches;
    std::vector<Span> written;
    std::vector<int64_t> sizes, offsets;
    int64_t partition = 0, workspace = 0, at = 0;
    int32_t max_group = 0;
    Batch open;
    std::vector<int32_t> small;
    int64_t few = 0;
    bool any_large = false;
    for (int32_t i = 0; i < n; ++i) {
        if (rows[i] < 0 || rows[i] > kMaxSide || cols[i] < 0 || cols[i] > kMaxSide)
            return bad(FP_ERR_RANGE, "matrix %d: %lld x %lld, sides go up to %lld", i, (long long)rows[i], (long long)cols[i],
                       (long long)kMaxSide);
        MuonRec& r = recs[(size_t)i];
        std::memset(&r, 0, sizeof r);
        if (group != nullptr) {
            if (group[i] < 0 || group[i] >= FP_MAX_GROUPS)
                return bad(FP_ERR_RANGE, "matrix %d: group %d outside [0, %d)", i, group[i], FP_MAX_GROUPS);
            r.group = group[i];
            max_group = std::max(max_group, group[i]);
        }
        const int64_t numel = rows[i] * cols[i];
        sizes.push_back(numel);
        offsets.push_back(partition);
        r.offset = partition;
        r.rows = (int32_t)rows[i];
        r.cols = (int32_t)cols[i];
        if (numel > 0) {
            auto place = [&](void* p, int64_t size, const char* what) -> fp_status {
                if (p == nullptr) return bad(FP_ERR_INVALID, "%s[%d] is NULL", what, i);
                if (!on(p, (uintptr_t)size)) return bad(FP_ERR_ALIGN, "%s[%d] misaligned", what, i);
                written.push_back(span_of(p, numel * size));
                return FP_OK;
            };
            fp_status st = FP_OK;
            if (master != nullptr) {
                if ((st = place(master[i], 4, "master")) != FP_OK) return st;
                r.master = master[i];
            }
            if (copies != nullptr) {
                if ((st = place(copies[i], 2, "copies")) != FP_OK) return st;
                r.copy = copies[i];
            }
            if (updates != nullptr) {
                if ((st = place(updates[i], dtype_bytes(update_dtype), "updates")) != FP_OK) return st;
                r.update = updates[i];
            }
            r.rp = (int32_t)pad64(rows[i]);
            r.cp = (int32_t)pad64(cols[i]);
            r.chunk = std::max<int64_t>(kChunk, ceil_div64(ceil_div64(numel, kMaxChunks), 1024) * 1024);
            r.chunks = (int32_t)ceil_div64(numel, r.chunk);
            partition += ceil_div64(numel, 32) * 32;
            if (ceil_div64(r.rp, kCastRows) * ceil_div64(r.cp, kCastCols) > 0xFFFFFFFFLL / 256)
                return bad(FP_ERR_RANGE, "matrix %d needs more workgroups than one launch holds", i);
            if (is_small(rows[i], cols[i])) ++few;
            else any_large = true;
        }
    }
    // A few small matrices beside a large one: its launches have room for them, and
    // one of their own would come on top.  Five steps of ragged matrices, together and
    // apart: 24 of 1 to 1448, 15 of them small, 205 and 248 us; 64 of 1 to 512, 61 small,
    // 128 and 182; 128 of 1 to 1448, 101 small, 319 and 344; 128 of 1 to 2048, 93 small,
    // 540 and 494.  Beside one large matrix they mostly pay up to about 32 (3000 x 3000 with
    // 32 of 128 x 128: 886 and 931; 1400 x 1300 with 32 of 160 x 160 260 and 299, of 32 x 48
    // 272 and 231; 1000 x 1000 with 64 of 128 x 128: 244 and 219), and not where its tiles
    // just fill the CUs (4096 x 4096 with 8 of 32 x 48: 1550 and 1467, with 128: 2101 and
    // 1469).
    const bool apart = !any_large || few > kFewSmall;
    for (int32_t i = 0; i < n; ++i) {
        MuonRec& r = recs[(size_t)i];
        if (r.rows > 0 && r.cols > 0) {
            if (apart && is_small(r.rows, r.cols)) {
                small.push_back(i);
            } else {
                open.mats.push_back(i);
                at = lay_out(&r, at);
                workspace = std::max(workspace, at);
            }
        }
        if (at >= kBatchBytes || (i + 1 == n && at > 0)) {
            close_batch(&recs, &open, &at, &table);
            workspace = std::max(workspace, at);
            batches.push_back(std::move(open));
            open = Batch();
            at = 0;
        }
    }
    std::vector<Small> smalls = group_small(recs, std::move(small), &table);
    std::sort(written.begin(), written.end());
    for (size_t i = 1; i < written.size(); ++i)
        if (meet(written[i - 1], written[i])) return bad(FP_ERR_INVALID, "two of the weights, copies and updates overlap");
    written = joined(std::move(written));
    std::vector<Span> read;
    fp_status st = check_grads(sizes, grad_dtype, written, grads, &read);
    if (st != FP_OK) return st;

    fp_muon* p = new fp_muon();
    p->n = n;
    p->grad_dtype = grad_dtype;
    p->copy_dtype = copy_dtype;
    p->update_dtype = update_dtype;
    p->has_master = master != nullptr;
    p->has_update = updates != nullptr;
    p->max_group = max_group;
    p->partition = partition;
    p->workspace = workspace;
    p->numel = std::move(sizes);
    p->offset = std::move(offsets);
    p->batches = std::move(batches);
    p->smalls = std::move(smalls);
    p->written = std::move(written);
    p->read = std::move(read);
    const size_t rec_b = sizeof(MuonRec) * (size_t)n, ptr_b = sizeof(void*) * (size_t)((n + 1) / 2 * 2);
    const size_t tile_b = sizeof(MatTile) * table.size();
    hipError_t e = hipGetDevice(&p->device);
    if (e == hipSuccess) e = hipMalloc(&p->dev, rec_b + ptr_b + tile_b);
    char* dev = static_cast<char*>(p->dev);
    if (e == hipSuccess) e = hipMemcpy(dev, recs.data(), rec_b, hipMemcpyHostToDevice);
    if (e == hipSuccess) e = hipMemcpy(dev + rec_b, grads, sizeof(void*) * (size_t)n, hipMemcpyHostToDevice);
    if (e == hipSuccess && tile_b > 0) e = hipMemcpy(dev + rec_b + ptr_b, table.data(), tile_b, hipMemcpyHostToDevice);
    if (e != hipSuccess) {
        free_plan(p);
        return device_error(e, "building the muon tables");
    }
    *out = p;
    return FP_OK;
}

fp_status set_grads(fp_muon* p, const void* const* grads, void* stream) {
    if (p == nullptr || grads == nullptr) return bad(FP_ERR_INVALID, "muon or grads is NULL");
    fp_status st = check_device(p);
    if (st != FP_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
    hipError_t e = hipStreamIsCapturing(s, &capture);
    if (e != hipSuccess) return device_error(e, "hipStreamIsCapturing");
    if (capture != hipStreamCaptureStatusNone)
        return bad(FP_ERR_INVALID, "the gradients cannot be changed while the stream is captured");
    std::vector<Span> read;
    if ((st = check_grads(p->numel, p->grad_dtype, p->written, grads, &read)) != FP_OK) return st;
    std::lock_guard<std::mutex> lock(p->mu);
    const size_t bytes = sizeof(void*) * (size_t)p->n;
    if (p->staging == nullptr) {
        if ((e = hipHostMalloc(&p->staging, bytes, hipHostMallocDefault)) != hipSuccess) {
            p->staging = nullptr;
            return device_error(e, "allocating the gradient table's staging");
        }
    }
    if (p->uploaded == nullptr) {
        if ((e = hipEventCreateWithFlags(&p->uploaded, hipEventDisableTiming)) != hipSuccess) {
            p->uploaded = nullptr;
            return device_error(e, "creating the upload event");
        }
    } else if ((e = hipEventSynchronize(p->uploaded)) != hipSuccess) {  // the staging may still feed the last upload
        return device_error(e, "hipEventSynchronize");
    }
    std::memcpy(p->staging, grads, bytes);
    if ((e = hipMemcpyAsync(p->grads(), p->staging, bytes, hipMemcpyHostToDevice, s)) != hipSuccess)
        return device_error(e, "uploading the gradient table");
    if ((e = hipEventRecord(p->uploaded, s)) != hipSuccess) return device_error(e, "hipEventRecord");
    p->read = std::move(read);
    return FP_OK;
}

// Momentum (may be null) and workspace: alignment, and no overlap with each
// other or with the plan's tensors.
fp_status check_buffers(fp_muon* p, const float* momentum, bool step, const void* workspace) {
    if (step && momentum == nullptr && p->partition > 0) return bad(FP_ERR_INVALID, "momentum is NULL");
    if (!on(momentum, 16)) return bad(FP_ERR_ALIGN, "momentum is not 16-byte aligned");
    if (workspace == nullptr && p->workspace > 0) return bad(FP_ERR_INVALID, "workspace is NULL");
    if (!on(workspace, 256)) return bad(FP_ERR_ALIGN, "workspace is not 256-byte aligned");
    std::lock_guard<std::mutex> lock(p->mu);
    const Span ws = span_of(workspace, p->workspace), mo = span_of(momentum, step ? 4 * p->partition : 0);
    if (meets_any(ws, p->written) || meets_any(ws, p->read)) return bad(FP_ERR_INVALID, "workspace overlaps one of the plan's tensors");
    if (meet(ws, mo)) return bad(FP_ERR_INVALID, "workspace overlaps momentum");
    if (meets_any(mo, p->written) || meets_any(mo, p->read)) return bad(FP_ERR_INVALID, "momentum overlaps one of the plan's tensors");
    return FP_OK;
}

// One step of the iteration: its coefficients and scales.
struct Step {
    float a, b, c;
    MuonScale s;
};

// The largest power of two that keeps values up to `most` below 60000.
float scale_for(double most) { return (float)std::ldexp(1.0, (int)std::floor(std::log2(60000.0 / most))); }

// B's diagonal multiplies the unrounded X only where the later steps let what this
// puts into directions that X does not hold grow by no more than this (muon_kernels.hip).
constexpr double kWholeGrowth = 4.0;

// Bounds of what fp16 has to hold.  With s the largest singular value of X, no
// element of X passes s, none of A s^2, none of B the largest |b t + c t^2| for
// t in [0, s^2]; the next s is the largest |a x + b x^3 + c x^5| for x in [0, s].
// Both are taken at the ends and where the derivative is 0.  s starts at 1, the
// Frobenius norm, and 1/64 is added for the roundings.
fp_status plan_steps(int32_t steps, const double* coefs, std::vector<Step>* out) {
    if (steps < 1 || steps > FP_MUON_MAX_STEPS) return bad(FP_ERR_RANGE, "steps %d outside [1, %d]", steps, FP_MUON_MAX_STEPS);
    if (coefs == nullptr) return bad(FP_ERR_INVALID, "coefs is NULL");
    double s = 1.0;
    for (int32_t i = 0; i < steps; ++i) {
        const double a = coefs[3 * i], b = coefs[3 * i + 1], c = coefs[3 * i + 2];
        if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return bad(FP_ERR_RANGE, "coefs of step %d are not finite", i);
        s *= 1.0 + 1.0 / 64;
        Step t;
        t.a = (float)a; t.b = (float)b; t.c = (float)c;
        const double s2 = s * s;
        double top = std::fabs(s2 * (b + c * s2));
        if (c != 0.0) {
            const double x = -b / (2 * c);
            if (x > 0.0 && x < s2) top = std::max(top, std::fabs(x * (b + c * x)));
        }
        double next = std::fabs(s * (a + s2 * (b + c * s2)));
        auto at = [&](double t2) {  // x^2 where the polynomial may be largest
            if (t2 > 0.0 && t2 < s2) next = std::max(next, std::fabs(std::sqrt(t2) * (a + t2 * (b + c * t2))));
        };
        // a + 3 b t + 5 c t^2 = 0: one root from the sum of what has b's sign, the other, which a difference would
        // lose where c is small, from their product; what is not a number, or is infinite, is not taken
        const double disc = 9 * b * b - 20 * a * c;
        if (disc >= 0.0) {
            const double q = -0.5 * (3 * b + std::copysign(std::sqrt(disc), b));
            at(q / (5 * c));
            at(a / q);
        }
        // beyond these the fp32 sums and the fp16 scales leave their ranges
        if (!(s <= 256.0) || !(top <= 60000.0) || !(next <= 256.0))
            return bad(FP_ERR_RANGE, "coefs of step %d let singular values grow to %g", i, next);
        const float of_a = scale_for(s2);
        t.s.x = scale_for(s);
        t.s.b = scale_for(std::max(top, 1e-3));
        t.s.un_x = 1.0f / t.s.x;
        t.s.un_xx = t.s.un_x * t.s.un_x;
        t.s.un_a = 1.0f / of_a;
        t.s.un_bx = t.s.un_x / t.s.b;
        t.s.gram = of_a * t.s.un_xx;
        s = std::max(next, 1e-3);
        t.s.x_next = scale_for(s * (1.0 + 1.0 / 64));
        out->push_back(t);
    }
    double growth = 1.0;  // of a direction near 0, over the later steps
    for (int32_t i = steps - 1; i >= 0; --i) {
        (*out)[(size_t)i].s.whole = growth <= kWholeGrowth;
        growth *= std::max(1.0, std::fabs(coefs[3 * i]));
    }
    return FP_OK;
}

fp_status run(fp_muon* p, MuonArgs a, MuonMore more, const std::vector<Step>& steps, void* stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    a.recs = p->recs();
    more.grads = p->grads();
    more.grad_dtype = p->grad_dtype;
    a.copy_dtype = p->copy_dtype;
    a.update_dtype = p->update_dtype;
    auto over = [&](const Run& r) {
        a.tiles = p->tile_table() + r.first;
        a.n_tiles = (int32_t)r.n;
    };
    hipError_t e;
    if (!p->smalls.empty()) {
        MuonSteps it;
        std::memset(&it, 0, sizeof it);
        it.n = (int32_t)steps.size();
        for (size_t i = 0; i < steps.size(); ++i) {
            it.s[i] = steps[i].s;
            it.c[i][0] = steps[i].a;
            it.c[i][1] = steps[i].b;
            it.c[i][2] = steps[i].c;
        }
        for (const Small& m : p->smalls) {
            over(m.run);
            if ((e = launch_muon_small(a, more, it, m.tiles, m.lds, s)) != hipSuccess) return device_error(e, "small matrices' launch");
        }
    }
    for (const Batch& b : p->batches) {
        over(b.moment);
        if ((e = launch_muon_moment(a, more, s)) != hipSuccess) return device_error(e, "momentum launch");
        over(b.norm);
        if (b.norm.n > 0 && (e = launch_muon_norm(a, more.eps, s)) != hipSuccess) return device_error(e, "norm launch");
        over(b.cast);
        a.s = steps[0].s;
        if ((e = launch_muon_cast(a, more, s)) != hipSuccess) return device_error(e, "cast launch");
        for (size_t i = 0; i < steps.size(); ++i) {
            a.s = steps[i].s;
            a.ca = steps[i].a;
            a.cb = steps[i].b;
            a.cc = steps[i].c;
            a.step = (int32_t)i;
            over(b.gram);
            if ((e = launch_muon_gram(a, b.gram_shape, s)) != hipSuccess) return device_error(e, "product launch");
            over(b.join);
            if (b.join.n > 0 && (e = launch_muon_join(a, s)) != hipSuccess) return device_error(e, "slices' launch");
            over(b.half);
            if ((e = launch_muon_poly(a, b.half_shape, s)) != hipSuccess) return device_error(e, "product launch");
            over(b.full);
            if (i + 1 < steps.size()) e = launch_muon_next(a, b.full_shape, s);
            else e = launch_muon_last(a, more.momentum != nullptr ? &more : nullptr, b.full_shape, s);
            if (e != hipSuccess) return device_error(e, "product launch");
        }
    }
    return FP_OK;
}

// Of zeros the norm is eps, and fp64 has to hold its reciprocal.
fp_status check_eps(double eps) {
    return std::isnormal(eps) && eps > 0.0 ? FP_OK : bad(FP_ERR_RANGE, "eps must be positive, finite and not subnormal");
}

}  // namespace

extern "C" fp_status fp_muon_create(int32_t n, const int64_t* rows, const int64_t* cols, const int32_t* group,
                                    int32_t grad_dtype, const void* const* grads, float* const* master,
                                    int32_t copy_dtype, void* const* copies, int32_t update_dtype, void* const* updates,
                                    fp_muon** out) {
    return guarded([&] {
        return create(n, rows, cols, group, grad_dtype, grads, master, copy_dtype, copies, update_dtype, updates, out);
    });
}

extern "C" void fp_muon_destroy(fp_muon* muon) {
    if (muon != nullptr) free_plan(muon);
}

extern "C" fp_status fp_muon_info(const fp_muon* muon, int64_t* partition, int64_t* workspace_bytes) {
    if (muon == nullptr) return bad(FP_ERR_INVALID, "muon is NULL");
    if (partition) *partition = muon->partition;
    if (workspace_bytes) *workspace_bytes = muon->workspace;
    return FP_OK;
}

extern "C" fp_status fp_muon_offsets(const fp_muon* muon, int64_t* offsets) {
    if (muon == nullptr || offsets == nullptr) return bad(FP_ERR_INVALID, "muon or offsets is NULL");
    std::copy(muon->offset.begin(), muon->offset.end(), offsets);
    return FP_OK;
}

extern "C" fp_status fp_muon_set_grads(fp_muon* muon, const void* const* grads, void* stream) {
    return guarded([&] { return set_grads(muon, grads, stream); });
}

extern "C" fp_status fp_muon_orthogonalize(fp_muon* muon, int32_t steps, const double* coefs, double eps, void* workspace,
                                           void* stream) {
    return guarded([&]() -> fp_status {
        if (muon == nullptr) return bad(FP_ERR_INVALID, "muon is NULL");
        if (!muon->has_update) return bad(FP_ERR_INVALID, "muon plan has no updates");
        std::vector<Step> it;
        fp_status st = plan_steps(steps, coefs, &it);
        if (st != FP_OK || (st = check_eps(eps)) != FP_OK) return st;
        if ((st = check_buffers(muon, nullptr, false, workspace)) != FP_OK) return st;
        if ((st = check_device(muon)) != FP_OK) return st;
        MuonArgs a;
        MuonMore more;
        std::memset(&a, 0, sizeof a);
        std::memset(&more, 0, sizeof more);
        a.ws = static_cast<char*>(workspace);
        more.eps = eps;
        return run(muon, a, more, it, stream);
    });
}

extern "C" fp_status fp_muon_step(fp_muon* muon, int32_t n_groups, const fp_muon_hparams* hp, int32_t steps,
                                  const double* coefs, double eps, float* momentum, const int32_t* found_inf,
                                  const double* grad_coef, void* workspace, void* stream) {
    return guarded([&]() -> fp_status {
        if (muon == nullptr) return bad(FP_ERR_INVALID, "muon is NULL");
        if (!muon->has_master) return bad(FP_ERR_INVALID, "muon plan has no master weights");
        if (n_groups <= muon->max_group || n_groups > FP_MAX_GROUPS)
            return bad(FP_ERR_RANGE, "n_groups %d: the matrices use groups up to %d, at most %d", n_groups, muon->max_group,
                       FP_MAX_GROUPS);
        if (hp == nullptr) return bad(FP_ERR_INVALID, "hparams is NULL");
        MuonArgs a;
        MuonMore more;
        std::memset(&a, 0, sizeof a);
        std::memset(&more, 0, sizeof more);
        for (int32_t g = 0; g < n_groups; ++g) {
            const fp_muon_hparams& h = hp[g];
            if (!std::isfinite(h.lr) || !std::isfinite(h.weight_decay) || !(h.beta >= 0.0 && h.beta < 1.0))
                return bad(FP_ERR_RANGE, "group %d: lr and weight_decay must be finite, beta in [0, 1)", g);
            if (h.adjust < FP_MUON_ADJUST_NONE || h.adjust > FP_MUON_ADJUST_SHAPE)
                return bad(FP_ERR_INVALID, "group %d: unknown adjust %d", g, h.adjust);
            more.g[g] = {h.lr, h.beta, 1.0 - h.lr * h.weight_decay, h.nesterov != 0, h.adjust};
        }
        std::vector<Step> it;
        fp_status st = plan_steps(steps, coefs, &it);
        if (st != FP_OK || (st = check_eps(eps)) != FP_OK) return st;
        if (!on(found_inf, 4)) return bad(FP_ERR_ALIGN, "found_inf misaligned");
        if (!on(grad_coef, 8)) return bad(FP_ERR_ALIGN, "grad_coef misaligned");
        if ((st = check_buffers(muon, momentum, true, workspace)) != FP_OK) return st;
        if ((st = check_device(muon)) != FP_OK) return st;
        a.ws = static_cast<char*>(workspace);
        a.found_inf = found_inf;
        more.eps = eps;
        more.momentum = momentum;
        more.g_coef = grad_coef;
        return run(muon, a, more, it, stream);
    });
}
