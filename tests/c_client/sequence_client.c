/*
 * sequence_client.c -- a plain C (C11) client of the sequence and search operators, built against the
 * headers in include/ only. It needs no GPU: it prints the argument struct sizes and some field offsets
 * as this C compiler lays them out next to the library's own sizes, and the status codes of calls that the
 * host-side checks refuse before any CUDA work (the device addresses are aligned and never dereferenced).
 */
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "gdn_beam.h"
#include "mamba_scan.h"

static void *at(int i) { return (void *)(((uintptr_t)1 << 40) + ((uintptr_t)i << 32)); }

static mamba_scan_args scan(void)
{
    mamba_scan_args m;
    memset(&m, 0, sizeof m);
    m.T = 300; m.S = 1; m.D = 64; m.N = 16; m.in_dtype = m.out_dtype = GDN_BF16;
    m.x = at(0); m.dt = at(1); m.A = at(2); m.Bm = at(3); m.Cm = at(4); m.y = at(5); m.h_last = at(6);
    m.x_stride = m.dt_stride = m.y_stride = 64;
    m.B_stride = m.C_stride = 16;
    m.num_states = 1;
    return m;
}

int main(void)
{
    printf("version %d\n", gdn_abi_version());
    printf("c_sizes %zu %zu %zu %zu %zu\n", sizeof(mamba_scan_args), sizeof(mamba_scan_grad_args), sizeof(gdn_beam_select_args),
           sizeof(gdn_beam_reorder_args), sizeof(gdn_beam_pool));
    printf("lib_sizes %zu %zu %zu %zu %zu\n", gdn_abi_struct_size(6), gdn_abi_struct_size(7), gdn_abi_struct_size(8),
           gdn_abi_struct_size(10), gdn_abi_struct_size(11));
    printf("offsets %zu %zu %zu %zu %zu %zu\n", offsetof(mamba_scan_args, num_states), offsetof(mamba_scan_args, err_flags),
           offsetof(mamba_scan_grad_args, dh0), offsetof(gdn_beam_select_args, eos_token), offsetof(gdn_beam_reorder_args, slots),
           offsetof(gdn_beam_pool, slot_bytes));

    mamba_scan_args m = scan();
    printf("scan_null %d\n", mamba_selective_scan(NULL, NULL));
    m.N = 129;
    printf("scan_bad_N %d\n", mamba_selective_scan(&m, NULL));
    m = scan();
    printf("scan_no_workspace %d\n", mamba_selective_scan(&m, NULL));

    mamba_scan_grad_args g;
    memset(&g, 0, sizeof g);
    g.s = scan();
    g.dy = at(7); g.dy_stride = 64;
    g.dz = at(8); g.dz_stride = 64;
    printf("dz_without_z %d\n", mamba_selective_scan_backward(&g, NULL));
    printf("workspace_grows %d\n", mamba_scan_workspace_bytes(300, 1, 64, 16, 1, 1) > mamba_scan_workspace_bytes(300, 1, 64, 16, 1, 0));

    gdn_beam_select_args b;
    memset(&b, 0, sizeof b);
    b.batch = 2; b.beams = 4; b.vocab = 1000; b.K = 4; b.logits_dtype = GDN_BF16; b.num_rows = 8; b.row_stride = 1000;
    b.logits = at(0); b.scores = at(1); b.out_scores = at(2); b.out_parents = at(3); b.out_tokens = at(4);
    printf("select_no_workspace %d\n", gdn_beam_select(&b, NULL));
    b.K = 65;
    printf("select_bad_K %d\n", gdn_beam_select(&b, NULL));

    gdn_beam_reorder_args r;
    const gdn_beam_pool pool = {at(0), 4096, 4096};
    memset(&r, 0, sizeof r);
    r.batch = 2; r.beams = 4; r.num_slots = 8; r.num_pools = 1; r.pools = &pool;
    r.slots = at(1); r.parents = at(2); r.new_slots = at(2);
    printf("reorder_over_parents %d\n", gdn_beam_reorder(&r, NULL));
    return 0;
}
