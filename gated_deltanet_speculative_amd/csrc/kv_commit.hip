// Commit of the paged caches for gfx950: the accepted path's rows of every layer moved together
// behind the committed ones, and the new lengths, as an all-or-nothing transaction.
//
// With the path a_0 < ... < a_m, row L + j takes row L + a_j.  Parents precede children, so
// a_j >= j, and a row that is written (L + j) is read only by the steps i <= j (a_i >= i): in
// ascending order, loads of a step before the stores of the same and later ones, the move is safe
// in place.  Each thread owns a 16-byte column of every row of one (lane, layer, K or V) and
// kv head: no other thread reads or writes it, so the order within the thread is enough.
//
// Bound by launch and by the dependent reads of the preflight (slot, length, page id) in front of
// the copies: every workgroup checks all lanes itself, as in the replay commit, so one launch decides.
#include "round_device.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

__global__ __launch_bounds__(kThreads) void kv_commit_kernel(AttnDims d, int n_layers, CacheLayers cl, PagedLanes l,
                                                             const int32_t *__restrict__ accept_node,
                                                             int32_t *__restrict__ new_len, int row_chunks) {
    __shared__ unsigned s_bitmap[kBitmapSlots / 32];
    __shared__ int s_word, s_bits;
    __shared__ uint32_t s_src[GDN_MAX_NODES], s_dst[GDN_MAX_NODES];  // cache rows of kv head 0
    const int tid = threadIdx.x, lane = tid & 63, c = blockIdx.y, side = blockIdx.x;
    const bool lengths = side == 2 * n_layers;  // the last workgroup of lane 0 writes the lengths
    if (lengths && c != 0) return;

    // ---- preflight over every lane
    const int st_in = *l.status;
    if (tid == 0) s_bits = 0;
    const LaneSlotsT<kThreads> slots(l.slot_ids, d.C);
    int bits = slot_preflight<kThreads>(slots, l.slot_ids, d.C, d.P, s_bitmap, &s_word);  // (has barriers)
    for (int t = tid; t < d.C; t += kThreads) {
        const Lane ln = paged_lane(d, l, t);
        if (ln.slot == -1) continue;
        bits |= ln.bits;
        const int e = accept_node[t];
        if (e < -1 || e >= min(max(ln.nodes, 0), d.N)) bits |= GDN_STATUS_ACCEPT;
    }
    if (l.parents)
        for (int k = tid; k < d.C * d.N; k += kThreads) {
            const int t = k / d.N, i = k - t * d.N;
            const Lane ln = paged_lane(d, l, t);
            if (ln.slot == -1 || ln.bits || i >= ln.nodes) continue;
            const int par = l.parents[k];
            if (par < -1 || par >= i) bits |= GDN_STATUS_PARENT;
            const int pid = l.page_table[(int64_t)ln.slot * d.max_pages + d.page((uint32_t)(ln.len + i))];
            if ((unsigned)pid >= (unsigned)d.n_pages) bits |= GDN_STATUS_PAGE;
        }
    if (bits) atomicOr(&s_bits, bits);
    __syncthreads();
    bits = s_bits;
    const bool commit = st_in == 0 && bits == 0;
    if (bits && tid == 0 && side == 0) atomicOr(l.status, bits);

    if (lengths) {
        for (int s = tid; s < d.P; s += kThreads) new_len[s] = l.seq_len[s];
        if (!commit) return;
        __syncthreads();  // (the same addresses are written again below)
        __threadfence_block();
        for (int t0 = 0; t0 < d.C; t0 += kThreads / 64) {  // a wave per lane
            const int t = t0 + (tid >> 6);
            if (t >= d.C) continue;
            const int s = l.slot_ids[t], e = accept_node[t];
            if (s == -1 || e < 0) continue;
            int n = e + 1;
            if (l.parents) {
                bool bad;
                const unsigned anc = tree_ancestors(l.parents + (int64_t)t * d.N, min(e + 1, d.N), bad);
                n = __popc(__shfl(anc, e));
            }
            if (lane == 0) new_len[s] = l.seq_len[s] + n;
        }
        return;
    }

    const int e = accept_node[c];
    const Lane ln = paged_lane(d, l, c);
    if (!commit || ln.slot == -1 || e < 0 || !l.parents) return;
    bool bad;
    const unsigned path = __shfl(tree_ancestors(l.parents + (int64_t)c * d.N, e + 1, bad), e);
    const int n = __popc(path);
    if (path == (n == 32 ? ~0u : (1u << n) - 1u)) return;  // the first n nodes: every row is in its place
    if (tid < n) {
        unsigned p = path;  // node a_tid: the tid-th set bit
        for (int j = 0; j < tid; ++j) p &= p - 1u;
        const uint32_t src = ln.len + __builtin_ctz(p), dst = ln.len + tid;
        const int32_t *table = l.page_table + (int64_t)ln.slot * d.max_pages;
        s_src[tid] = cache_row(d, table[d.page(src)], 0, src, d.page(src));
        s_dst[tid] = cache_row(d, table[d.page(dst)], 0, dst, d.page(dst));
    }
    __syncthreads();
    v4i *cache = static_cast<v4i *>(side < n_layers ? cl.k[side] : cl.v[side - n_layers]);
    const size_t head = (size_t)d.page.d * row_chunks;  // 16-byte chunks between the heads of a page
    const int first = __builtin_ctz(~path);             // rows in front of the first gap stay
    for (int col = tid; col < d.Hkv * row_chunks; col += kThreads) {
        v4i *p = cache + (col / row_chunks) * head + col % row_chunks;
        constexpr int kAhead = 4;  // loads in flight; a row written by these steps is read by none behind them
        for (int j0 = first; j0 < n; j0 += kAhead) {
            v4i v[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (j0 + j < n) v[j] = p[(size_t)s_src[j0 + j] * row_chunks];
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (j0 + j < n) p[(size_t)s_dst[j0 + j] * row_chunks] = v[j];
        }
    }
}

}  // namespace

hipError_t launch_kv_commit(const AttnDims &d, int n_layers, const CacheLayers &cl, const PagedLanes &l,
                            const int32_t *accept_node, int32_t *new_len, hipStream_t stream) {
    const int es = d.dtype == GDN_DTYPE_F32 ? 4 : 2;
    // without parents no row moves: only the workgroup that writes the lengths is launched
    const int layers = l.parents ? n_layers : 0;
    hipLaunchKernelGGL(kv_commit_kernel, dim3(2 * layers + 1, l.parents ? d.C : 1), dim3(kThreads), 0, stream, d, layers,
                       cl, l, accept_node, new_len, d.D * es / 16);
    return hipGetLastError();
}

}  // namespace gdn
