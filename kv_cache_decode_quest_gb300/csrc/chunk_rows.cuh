// The rows of a chunk of new tokens as the kernels that append them see them: which rows
// have a place in the cache, which rows of a sequence lie in one page (a piece, the work of
// one warp, which then owns that page's summary), and which row sets a sequence's length.
#pragma once

#include "common.cuh"

namespace se {
namespace {

// Row t of a chunk: slot is -1 where it has none, where it is dropped (`bad`: the slot
// is outside the pages, or seq or pos outside the block table) and past the arrays.
struct ChunkRow {
    int slot, pos, seq;
    bool bad;
};
__device__ __forceinline__ ChunkRow chunk_row(const se_paged_kv& kv, const se_chunk& ck, int batch,
                                              int t) {
    ChunkRow r = {-1, -1, -1, false};
    if (t < 0 || t >= ck.max_tokens) return r;
    r.slot = ck.slot[t];
    r.pos = ck.pos[t];
    r.seq = ck.seq[t];
    r.bad = r.slot != -1 &&
            (r.slot < 0 || r.slot / kPage >= kv.num_pages || r.seq < 0 || r.seq >= batch ||
             r.pos < 0 || r.pos / kPage >= kv.max_pages_per_seq ||
             r.pos % kPage != r.slot % kPage);
    if (r.bad) {
        r.slot = -1;
        if (r.seq == -1) r.seq = -2;                // names none, but is no row past the last sequence
    }
    return r;
}

// Lengths: each sequence's last row with a slot sets ctx_len, and no other row writes it.
// Lane l holds row t of 32; lanes 1..16 hold the rows this warp answers for.  The row after
// such a row tells, unless that one has no slot (a page that was not found, a dropped
// row): then the warp looks on, past rows without a slot that are the same sequence's or
// name none that exists, 32 at a time, to the next row that decides.
__device__ __forceinline__ void commit_lengths(const se_paged_kv& kv, const se_chunk& ck, int batch,
                                               int t, int lane, const ChunkRow& row) {
    const bool mine = row.slot >= 0 && lane >= 1 && lane <= kPage;
    const int nslot = __shfl_down_sync(0xffffffffu, row.slot, 1);
    const int nseq = __shfl_down_sync(0xffffffffu, row.seq, 1);
    auto passes = [&](int s, int b) { return s == b || s < -1 || s >= batch; };
    const bool hole = mine && nslot < 0 && passes(nseq, row.seq);
    if (mine && !hole && (nslot < 0 || nseq != row.seq)) kv.ctx_len[row.seq] = row.pos + 1;
    for (uint32_t m = __ballot_sync(0xffffffffu, hole); m != 0; m &= m - 1) {
        const int f = __ffs(m) - 1;
        const int b = __shfl_sync(0xffffffffu, row.seq, f);
        const int len = __shfl_sync(0xffffffffu, row.pos, f) + 1;
        uint32_t more, end;                         // rows that go on, rows that are another's or none's
        for (int r = __shfl_sync(0xffffffffu, t, f) + 1;; r += 32) {
            const ChunkRow x = chunk_row(kv, ck, batch, r + lane);
            more = __ballot_sync(0xffffffffu, x.slot >= 0 && x.seq == b);
            end = __ballot_sync(0xffffffffu,
                                x.slot >= 0 ? x.seq != b : !passes(x.seq, b));
            if ((more | end) != 0) break;           // (rows past max_tokens end it)
        }
        if (lane == 0 && __ffs(more | end) == __ffs(end)) kv.ctx_len[b] = len;
    }
}

// Rows of a piece: slot and position go with the row, d rows behind the first.
__device__ __forceinline__ bool same_piece(int d, int slot_d, int pos_d, int seq_d, int slot0,
                                           int pos0, int seq0) {
    return slot_d >= 0 && seq_d == seq0 && slot_d - slot0 == d && pos_d - pos0 == d &&
           pos_d / kPage == pos0 / kPage;
}

// The pieces that begin in rows [16 group, 16 group + 16), found by each warp from the slots of the 32
// rows around them (ballots).
struct Pieces {
    ChunkRow row;            // of row t
    int t;                   // lane l looks at row 16 group - 1 + l
    uint32_t lead;           // bit l: a piece begins with lane l's row
};
__device__ __forceinline__ Pieces find_pieces(const se_paged_kv& kv, const se_chunk& ck, int batch,
                                              int group, int lane) {
    Pieces p;
    const int t = p.t = group * kPage - 1 + lane;
    p.row = chunk_row(kv, ck, batch, t);
    const int slot = p.row.slot, pos = p.row.pos, seq = p.row.seq;
    const bool valid = slot >= 0;
    const int pslot = __shfl_up_sync(0xffffffffu, slot, 1);
    const int pseq = __shfl_up_sync(0xffffffffu, seq, 1);
    const int ppos = __shfl_up_sync(0xffffffffu, pos, 1);
    const bool begins = valid && lane >= 1 && lane <= kPage &&
                        !(pslot >= 0 && pseq == seq && ppos + 1 == pos && pslot + 1 == slot &&
                          pos % kPage != 0);
    uint32_t lead_m = __ballot_sync(0xffffffffu, begins);
    // behind rows without a slot a page may have begun before them: up to 15 rows back
    const bool unsure = begins && pslot < 0 && t > 0 && pos % kPage != 0 &&
                        (pseq == seq || pseq < 0 || pseq >= batch);
    uint32_t look = __ballot_sync(0xffffffffu, unsure);
    if (look != 0) {
        const ChunkRow far = chunk_row(kv, ck, batch, t - 32);
        for (; look != 0; look &= look - 1) {
            const int f = __ffs(look) - 1;
            const int slot0 = __shfl_sync(0xffffffffu, slot, f);
            const int pos0 = __shfl_sync(0xffffffffu, pos, f);
            const int seq0 = __shfl_sync(0xffffffffu, seq, f);
            if (__any_sync(0xffffffffu,
                           (lane < f && same_piece(lane - f, slot, pos, seq, slot0, pos0, seq0)) ||
                               same_piece(lane - 32 - f, far.slot, far.pos, far.seq, slot0, pos0,
                                          seq0)))
                lead_m &= ~(1u << f);
        }
    }
    p.lead = lead_m;
    return p;
}

// Piece i of them: the lane of its first row, that row, and (bit r) which rows behind it are of the piece.
struct Piece {
    int f, slot0, pos0, seq0;
    uint32_t rows;
};
__device__ __forceinline__ Piece piece_at(const Pieces& p, int i, int lane) {
    uint32_t rest = p.lead;
    for (; i > 0; --i) rest &= rest - 1;
    Piece q;
    q.f = __ffs(rest) - 1;
    q.slot0 = __shfl_sync(0xffffffffu, p.row.slot, q.f);
    q.pos0 = __shfl_sync(0xffffffffu, p.row.pos, q.f);
    q.seq0 = __shfl_sync(0xffffffffu, p.row.seq, q.f);
    q.rows = __ballot_sync(0xffffffffu, same_piece(lane - q.f, p.row.slot, p.row.pos, p.row.seq,
                                                   q.slot0, q.pos0, q.seq0)) >> q.f;
    return q;
}

}  // namespace
}  // namespace se
