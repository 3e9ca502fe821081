"""What the cross entropy's C calls take and refuse before any device work (no GPU)."""
import vocab_selected_token_tile_gb300 as rlk


def contract(**kw):
    base = dict(T=8, V=1000, H=64)
    base.update(kw)
    return rlk.LinearCeContract(**base)


def test_no_rows_need_no_output(built):
    # a frozen head's step of an empty batch: its dhidden has no element and so no address
    assert rlk.rlk_linear_ce_bwd(contract(T=0), *[None] * 10) == rlk.RLK_OK
    assert rlk.rlk_linear_ce_bwd(contract(T=1), *[None] * 10) == rlk.RLK_ERR_INVALID_ARG


def test_overlaps_are_refused(built):
    c = contract(reduction=rlk.REDUCE_NONE)
    step = 1 << 20  # above every operand's bytes

    def refused(call, args, names, outputs):
        for out in outputs:
            for other in range(len(args)):
                if other == out:
                    continue
                moved = list(args)
                moved[out] = args[other] + 16  # inside the other's 32 bytes at least
                if names[other] == "active_mask":
                    moved[out] = args[other]  # 8 bytes
                assert call(c, *moved, None) == rlk.RLK_ERR_INVALID_ARG, (names[out], names[other])
                message = rlk.rlk_last_error_message()
                assert "overlaps" in message and names[out] in message and names[other] in message
    fwd = ["hidden", "weight", "targets", "active_mask", "loss", "lse", "workspace"]
    refused(rlk.rlk_linear_ce_fwd, [step * (i + 1) for i in range(7)], fwd, (4, 5, 6))
    bwd = ["hidden", "weight", "targets", "active_mask", "lse", "grad_loss", "dhidden", "dweight", "workspace"]
    refused(rlk.rlk_linear_ce_bwd, [step * (i + 1) for i in range(9)], bwd, (6, 7, 8))
