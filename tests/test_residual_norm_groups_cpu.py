"""The backward pass's workspace has room for as many workgroups as each type pair's
launch wants: fp32 branches have 8 waves to a workgroup, others 12."""
import muon_newton_schulz_step_amd as mn


def groups(rows, teams):
    """As few workgroups as give no team more rows than 256 of them would."""
    all_ = -(-rows // teams)
    each = -(-all_ // 256)
    return -(-all_ // each)


def test_room_for_every_type():
    # (columns, waves of a team, waves of a workgroup by branch type: bf16, fp32)
    for cols, team, waves in ((512, 1, (12, 8)), (1024, 2, (12, 8)), (1536, 3, (12, 6)), (2048, 4, (12, 8))):
        for rows in (1, 7, 100, 512, 1500, 2048, 2100, 5000, 100_000):
            most = max(groups(rows, w // team) for w in waves)
            need = -(-most * 8 // 256) * 256 + most * 4 * cols * 4
            assert mn.residual_norm_backward_workspace_bytes(rows, cols, True) >= need
