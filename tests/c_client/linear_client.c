/*
 * linear_client.c -- a plain C (C11) client of linear attention and rotary positions, built against the headers in
 * include/ only. It needs no GPU: struct sizes and offsets as this compiler lays them out next to the library's, and the status
 * codes of calls that the host-side checks refuse before any CUDA work (the device addresses are never dereferenced).
 */
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "gdn_linear.h"
#include "gdn_rotary.h"

static void *at(int i) { return (void *)(((uintptr_t)1 << 40) + ((uintptr_t)i << 32)); }

static gdn_linear_args attention(void)
{
    gdn_linear_args a;
    memset(&a, 0, sizeof a);
    a.T = 4096; a.S = 1; a.H = 2; a.HV = 4; a.K = 64; a.V = 64; a.in_dtype = a.out_dtype = GDN_BF16;
    a.q = at(0); a.k = at(1); a.v = at(2); a.g = at(3); a.o = at(4);
    a.q_stride = a.k_stride = 128; a.v_stride = a.o_stride = 256; a.g_stride = 4;
    a.q_head_stride = a.k_head_stride = a.v_head_stride = a.o_head_stride = 64;
    return a;
}

int main(void)
{
    printf("version %d\n", gdn_abi_version());
    printf("c_sizes %zu %zu %zu %zu\n", sizeof(gdn_linear_args), sizeof(gdn_linear_grad_args), sizeof(gdn_linear_step_args),
           sizeof(gdn_rotary_args));
    printf("lib_sizes %zu %zu %zu %zu\n", gdn_abi_struct_size(12), gdn_abi_struct_size(13), gdn_abi_struct_size(14),
           gdn_abi_struct_size(15));
    printf("offsets %zu %zu %zu %zu\n", offsetof(gdn_linear_args, workspace), offsetof(gdn_linear_grad_args, d_o),
           offsetof(gdn_linear_step_args, state), offsetof(gdn_rotary_args, magnitude));

    gdn_linear_args a = attention();
    printf("attention_null %d\n", gdn_linear_attention(NULL, NULL));
    printf("attention_no_workspace %d\n", gdn_linear_attention(&a, NULL));
    a.K = 48;
    printf("attention_bad_K %d\n", gdn_linear_attention(&a, NULL));
    a = attention();
    a.HV = 3;
    printf("attention_bad_heads %d\n", gdn_linear_attention(&a, NULL));

    gdn_linear_grad_args g;
    memset(&g, 0, sizeof g);
    g.s = attention();
    printf("gradient_no_d_o %d\n", gdn_linear_attention_backward(&g, NULL));
    printf("workspace_grows %d\n", gdn_linear_workspace_bytes(4096, 1, 2, 4, 64, 64, GDN_BF16, 1, 1) >
                                       gdn_linear_workspace_bytes(4096, 1, 2, 4, 64, 64, GDN_BF16, 1, 0));

    gdn_linear_step_args s;
    memset(&s, 0, sizeof s);
    printf("step_null %d\n", gdn_linear_attention_step(NULL, NULL, -1, NULL));
    printf("step_empty %d\n", gdn_linear_attention_step(&s, NULL, -1, NULL));

    gdn_rotary_args r;
    memset(&r, 0, sizeof r);
    r.T = 3; r.H = 2; r.D = 64; r.rotary_dim = 33; r.dtype = GDN_BF16;
    r.q = r.q_out = at(0); r.positions = at(1); r.frequencies = at(2);
    r.q_stride = r.q_out_stride = 128; r.q_head_stride = r.q_out_head_stride = 64;
    printf("rotary_odd %d\n", gdn_rotary(&r, NULL));
    r.rotary_dim = 32;
    r.frequencies = NULL;
    printf("rotary_null %d\n", gdn_rotary(&r, NULL));
    return 0;
}
