// Index arithmetic of the paged key/value cache: where a token lives, which
// keys a query row sees, and how the work of one attn_paged_fwd call is cut
// into equal shares.  Plain integer code for host and device: the kernels use
// it and a host test checks it exhaustively, out-of-range input included.
//
// Work of a call.  A list entry's new tokens are cut into units of `tpu`
// tokens; a unit is (entry i, kv head h, token block u) and has tpu * g query
// rows (row r: token r / g of the block, query head h * g + r % g), so one
// stream over K and V of head h serves all g query heads that share it.  A
// unit runs over its visible keys in tiles of `tk`.  All units, ordered by
// (i, h, u), form one line; its length is measured in keys (plus a constant
// per unit) so that prefix sums have a closed form; CTA c of G takes the
// stretch [W c / G, W (c + 1) / G) and so may begin and end inside a unit.
// Lengths stay on the device: nothing here needs them on the host.
#pragma once

#ifdef __CUDACC__
#define ETA_HD __host__ __device__ __forceinline__
#else
#define ETA_HD inline
#endif

namespace eta {

struct PagedGeom {
    const int *page_table;   // [rows][max_pages]
    const int *seq_lens;     // [rows]
    const int *seqs;         // [n] table rows of the list, or null: 0 .. n-1
    const int *q_start;      // [n + 1] first new token of each entry
    const int *granted = nullptr;   // [n], or null: an entry with 0 takes no part
    int n, rows, max_pages, pages, page_size;
    int T, max_q;            // rows of Q; the most new tokens of an entry
    int heads, g;            // kv heads, query heads to each
    int causal;
    int tpu, tk;             // tokens per unit, keys per tile
    int unit_cost;           // a unit's fixed cost, in keys
    int min_share;           // the least work worth a CTA, in keys
    // derived (paged_derive): divisions are slow where a call takes microseconds
    int page_shift, tk_shift;   // page_size and tk are powers of two
    unsigned g_mul;             // r / g = r * g_mul >> 16 for r < 256
};

ETA_HD void paged_derive(PagedGeom &gm) {
    gm.page_shift = 0;
    while ((1 << gm.page_shift) < gm.page_size) ++gm.page_shift;
    gm.tk_shift = 0;
    while ((1 << gm.tk_shift) < gm.tk) ++gm.tk_shift;
    gm.g_mul = (65536u + static_cast<unsigned>(gm.g) - 1) / static_cast<unsigned>(gm.g);
}

// Row r < 256 of a unit: its token within the unit (r / g; the head is the rest).
ETA_HD int paged_token(const PagedGeom &gm, int r) { return static_cast<int>(static_cast<unsigned>(r) * gm.g_mul >> 16); }

// a / b, by the short division where both fit into 32 bits.
ETA_HD long long paged_div(long long a, long long b) {
    if (((a | b) >> 32) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
    return a / b;
}

// One entry of the list.  nq = 0: nothing to do (or a bad entry, or one that got no room).
struct PagedEntry {
    int seq, q0, nq, len;
};

// Reads entry i; returns false for one that is out of range (a table row, a
// token range or a length that does not fit), which then has nq = 0, or its
// length cut to what the table can hold.
ETA_HD bool paged_entry(const PagedGeom &gm, int i, PagedEntry &e) {
    const int seq = gm.seqs ? gm.seqs[i] : i;
    const int q0 = gm.q_start[i], q1 = gm.q_start[i + 1];
    e.seq = 0;
    e.q0 = 0;
    e.nq = 0;
    e.len = 0;
    if (gm.granted && gm.granted[i] == 0) return true;   // (left out on purpose)
    if (seq < 0 || seq >= gm.rows || q0 < 0 || q1 < q0 || q1 > gm.T || q1 - q0 > gm.max_q) return false;
    const int cap = gm.max_pages * gm.page_size;
    const int len = gm.seq_lens[seq];
    e.seq = seq;
    e.q0 = q0;
    e.nq = q1 - q0;
    e.len = len < 0 ? 0 : len > cap ? cap : len;
    return e.len == len;
}

// Keys that new token t of the entry sees (a prefix of the sequence): token t
// is at position len - nq + t.
ETA_HD int paged_visible(const PagedGeom &gm, const PagedEntry &e, int t) {
    if (!gm.causal) return e.len;
    const int v = e.len - e.nq + t + 1;
    return v < 0 ? 0 : v > e.len ? e.len : v;
}

ETA_HD int paged_units(const PagedGeom &gm, const PagedEntry &e) {
    return e.nq <= gm.tpu ? (e.nq > 0 ? 1 : 0) : (e.nq + gm.tpu - 1) / gm.tpu;
}

// Tiles of unit u: at least one, so that rows without any key are written.
ETA_HD int paged_tiles(const PagedGeom &gm, const PagedEntry &e, int u) {
    const int last = (u + 1) * gm.tpu < e.nq ? (u + 1) * gm.tpu : e.nq;
    const int keys = paged_visible(gm, e, last - 1);
    return keys <= gm.tk ? 1 : ((keys - 1) >> gm.tk_shift) + 1;
}

// Work of units [0, u) of one head, in keys (every unit before the last has
// tpu tokens; a causal unit is counted up to its last token's position).
ETA_HD long long paged_before(const PagedGeom &gm, const PagedEntry &e, int u) {
    const long long base = gm.causal ? (e.len > e.nq ? e.len - e.nq : 0) : e.len;
    const long long each = gm.unit_cost + base;
    return u * each + (gm.causal ? static_cast<long long>(gm.tpu) * u * (u + 1) / 2 : 0);
}
ETA_HD long long paged_head_work(const PagedGeom &gm, const PagedEntry &e) {
    const int U = paged_units(gm, e);
    if (U == 0) return 0;
    const long long base = gm.causal ? (e.len > e.nq ? e.len - e.nq : 0) : e.len;
    return paged_before(gm, e, U - 1) + gm.unit_cost + base + (gm.causal ? e.nq : 0);
}
ETA_HD long long paged_entry_work(const PagedGeom &gm, const PagedEntry &e) {
    return paged_head_work(gm, e) * gm.heads;
}

// A place on the line: before tile `tile` of unit (i, h, u).
struct PagedPos {
    int i, h, u, tile;
};
ETA_HD bool paged_less(const PagedPos &a, const PagedPos &b) {
    if (a.i != b.i) return a.i < b.i;
    if (a.h != b.h) return a.h < b.h;
    if (a.u != b.u) return a.u < b.u;
    return a.tile < b.tile;
}
ETA_HD void paged_next_unit(const PagedGeom &gm, const PagedEntry &e, PagedPos &p) {
    p.tile = 0;
    if (++p.u < paged_units(gm, e)) return;
    p.u = 0;
    if (++p.h < gm.heads) return;
    p.h = 0;
    ++p.i;
}

// The place at distance x (0 <= x < the entry's work) into entry i, moved to
// the nearest tile boundary.
ETA_HD PagedPos paged_locate(const PagedGeom &gm, const PagedEntry &e, int i, long long x) {
    const long long hw = paged_head_work(gm, e);
    PagedPos p;
    p.i = i;
    p.h = static_cast<int>(paged_div(x, hw));
    x -= p.h * hw;
    int lo = 0, hi = paged_units(gm, e) - 1;   // the last unit that begins at or before x
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (paged_before(gm, e, mid) <= x) lo = mid;
        else hi = mid - 1;
    }
    p.u = lo;
    x -= paged_before(gm, e, lo);
    const long long t = (x + gm.tk / 2) >> gm.tk_shift;
    const int tiles = paged_tiles(gm, e, lo);
    p.tile = t < tiles ? static_cast<int>(t) : tiles;
    if (p.tile == tiles) paged_next_unit(gm, e, p);
    return p;
}

// CTAs that get a share of W, and where share c begins.
ETA_HD int paged_shares(const PagedGeom &gm, long long W, int ctas) {
    const long long most = paged_div(W + gm.min_share - 1, gm.min_share);
    return most < 1 ? 1 : most < ctas ? static_cast<int>(most) : ctas;
}
ETA_HD long long paged_share_begin(long long W, int c, int shares) {
    if (c >= shares) return W;
    // W c / shares without overflow: W < 2^62, shares <= 4096
    const long long each = paged_div(W, shares);
    return each * c + paged_div((W - each * shares) * c, shares);
}

// The page of tile-relative page k of a tile that starts at key `key0` (a
// multiple of the page size, or inside one page): its id, or -1 where the
// table has no such column or the id is not a page of the pool.
ETA_HD int paged_page(const PagedGeom &gm, int seq, int col) {
    if (col < 0 || col >= gm.max_pages) return -1;
    const int id = gm.page_table[static_cast<long long>(seq) * gm.max_pages + col];
    return (id >= 0 && id < gm.pages) ? id : -1;
}

}  // namespace eta
